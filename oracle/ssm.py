"""The short causal convolution, the selective state space scan and the group norm in 64 bits, straight from the definitions
(torch, any device): token by token, the reverse modes written out by hand.

    s_t = bias + sum_j w_j x_{t-W+1+j},  y_t = s_t or silu(s_t)
    delta_t = softplus(dt_t + dt_bias),  h_t = e^{-e^{A_log} delta_t} h_{t-1} + delta_t x_t B_t,
    y_t = (C_t . h_t + D x_t) silu(z_t)

    n = (x - mean) / sqrt(var + eps) over positions and channels of a group,  y = w n + b or silu of it

x, dt, z [B, T, D], B, C [B, T, G, N], A_log [D, N]; channel d reads group d // (D // G).  With ``size=True`` every
factor and every summand is taken without its sign: the sum of the magnitudes that an output is made of, which its
rounding errors are proportional to.
"""
from __future__ import annotations

import math

import torch


def _f64(*xs):
    return [None if x is None else x.detach().double() for x in xs]


def _abs(size, *xs):
    return [x.abs() if size and x is not None else x for x in xs]


def _silu(x):
    return x / (1 + torch.exp(-x))


def _dsilu(x):
    s = 1 / (1 + torch.exp(-x))
    return s * (1 + x * (1 - s))


def _softplus(x):
    return torch.maximum(x, torch.zeros_like(x)) + torch.log1p(torch.exp(-x.abs()))


def _extended(x, state0, W):
    B, _, D = x.shape
    before = x.new_zeros(B, W - 1, D) if state0 is None else state0
    return torch.cat([before, x], 1)


def _taps(full, w, bias, T):
    s = full.new_zeros(full.shape[0], T, full.shape[2])
    for j in range(w.shape[1]):
        s = s + w[:, j] * full[:, j:j + T]
    return s if bias is None else s + bias


def conv(x, w, bias=None, state0=None, silu=True, size=False):
    """(y, the last W - 1 inputs)."""
    x, w, bias, state0 = _f64(x, w, bias, state0)
    T, W = x.shape[1], w.shape[1]
    full = _extended(x, state0, W)
    s = _taps(full, w, bias, T)
    y = _silu(s) if silu else s
    if size:  # silu has a slope of at most 1.1
        y = 1.1 * _taps(*_abs(True, full, w, bias), T)
    return y, full[:, T:]


def conv_bwd(x, w, bias, state0, dy, dstate_T=None, silu=True, size=False):
    x, w, bias, state0, dy, dstate_T = _f64(x, w, bias, state0, dy, dstate_T)
    T, W = x.shape[1], w.shape[1]
    full = _extended(x, state0, W)
    ds = dy
    if silu:  # the slope of silu' is at most 0.5
        s = _taps(full, w, bias, T)
        ds = dy * _dsilu(s)
        if size:
            ds = dy.abs() * (1.1 + 0.5 * _taps(*_abs(True, full, w, bias), T))
    full, w, ds, dstate_T = _abs(size, full, w, ds, dstate_T)
    dfull = torch.zeros_like(full)
    for j in range(W):
        dfull[:, j:j + T] += w[:, j] * ds
    if dstate_T is not None:
        dfull[:, T:] += dstate_T
    dw = torch.stack([(ds * full[:, j:j + T]).sum((0, 1)) for j in range(W)], 1)
    return {"dx": dfull[:, W - 1:], "dw": dw, "dbias": None if bias is None else ds.sum((0, 1)), "dstate0": dfull[:, :W - 1]}


def _scan_inputs(x, dt, A_log, B, C, D, dt_bias, z, S0, size):
    x, dt, A_log, B, C, D, dt_bias, z, S0 = _f64(x, dt, A_log, B, C, D, dt_bias, z, S0)
    rep = x.shape[2] // B.shape[2]
    arg = dt if dt_bias is None else dt + dt_bias
    delta, A = _softplus(arg), -torch.exp(A_log)
    S = x.new_zeros(x.shape[0], *A.shape) if S0 is None else S0
    D = x.new_zeros(x.shape[2]) if D is None else D
    x, B, C, D, S = _abs(size, x, B, C, D, S)
    return x, arg, delta, A, B.repeat_interleave(rep, 2), C.repeat_interleave(rep, 2), D, z, S


def scan(x, dt, A_log, B, C, D=None, dt_bias=None, z=None, S0=None, size=False, keep=False):
    """(y, S_T) [and, with `keep`, C . h and the state that every token starts from]."""
    x, _, delta, A, B, C, D, z, S = _scan_inputs(x, dt, A_log, B, C, D, dt_bias, z, S0, size)
    ys, kept = torch.zeros_like(x), []
    for t in range(x.shape[1]):
        kept.append(S)
        S = torch.exp(delta[:, t, :, None] * A) * S + (delta[:, t] * x[:, t])[..., None] * B[:, t]
        ys[:, t] = (S * C[:, t]).sum(-1)
    y = ys + D * x
    if z is not None:
        y = y * _abs(size, _silu(z))[0]
    return (y, S, ys, kept) if keep else (y, S)


def scan_bwd(x, dt, A_log, B, C, D, dt_bias, z, S0, dy, dS_T=None, size=False):
    """Gradients of any loss with dL/dy = dy and dL/dS_T = dS_T."""
    groups = B.shape[2]
    _, S_T, ys, kept = scan(x, dt, A_log, B, C, D, dt_bias, z, S0, size, keep=True)
    with_D, with_bias = D is not None, dt_bias is not None
    x, arg, delta, A, B, C, D, z, _ = _scan_inputs(x, dt, A_log, B, C, D, dt_bias, z, S0, size)
    dy, dS_T = _abs(size, *_f64(dy, dS_T))
    A = _abs(size, A)[0]
    out, g = {"dz": None}, dy
    if z is not None:
        # (without sign: silu' is rounded relative to the size of its parts, 1.1 at most)
        out["dz"] = dy * (ys + D * x) * (1.1 if size else _dsilu(z))
        g = dy * _abs(size, _silu(z))[0]
    decay = torch.exp(-delta[..., None] * torch.exp(A_log.detach().double()))
    lam = torch.zeros_like(S_T) if dS_T is None else dS_T
    dx, darg, dA = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(S_T)
    dB, dC = torch.zeros_like(B), torch.zeros_like(C)
    for t in range(x.shape[1] - 1, -1, -1):
        u = (delta[:, t] * x[:, t])[..., None]
        h = decay[:, t] * kept[t] + u * B[:, t]
        lam = lam + g[:, t][..., None] * C[:, t]
        dC[:, t], dB[:, t] = g[:, t][..., None] * h, lam * u
        du = (lam * B[:, t]).sum(-1)
        lam = lam * decay[:, t]
        w = lam * kept[t]
        dA = dA + w * delta[:, t][..., None]
        dx[:, t] = du * delta[:, t]
        darg[:, t] = (w * A).sum(-1) + du * x[:, t]
    ddt = darg / (1 + torch.exp(-arg))
    fold = lambda m: m.unflatten(2, (groups, -1)).sum(3)  # noqa: E731
    out |= {"dx": dx + D * g, "ddt": ddt, "dB": fold(dB), "dC": fold(dC), "dA_log": dA.sum(0) * A,
            "dD": (g * x).sum((0, 1)) if with_D else None, "ddt_bias": ddt.sum((0, 1)) if with_bias else None, "dS0": lam}
    return out


def _normed(x, groups, eps, stats=None):
    xg = x.reshape(x.shape[0], math.prod(x.shape[1:-1]), groups, x.shape[-1] // groups)
    if stats is not None:
        mean, r = (t[:, None, :, None] for t in stats.double().unbind(-1))
        return (xg - mean) * r, mean, r
    mean = xg.mean((1, 3), keepdim=True)
    r = 1 / torch.sqrt(((xg - mean) ** 2).mean((1, 3), keepdim=True) + eps)
    return (xg - mean) * r, mean, r


def group_norm(x, w, b, groups, eps=1e-5, silu=False, stats=None):
    """(y, stats) for x [rows, ..., C]; from given ``stats`` if there are."""
    x, w, b = _f64(x, w, b)
    n, mean, r = _normed(x, groups, eps, stats)
    s = n.reshape(x.shape)
    s = s if w is None else s * w
    s = s if b is None else s + b
    return _silu(s) if silu else s, torch.stack([mean[:, 0, :, 0], r[:, 0, :, 0]], -1)


def group_norm_bwd(x, w, b, groups, dy, eps=1e-5, silu=False, stats=None):
    """Gradients, and the sum of the magnitudes that each is made of; with ``stats`` taken for x's own."""
    x, w, b, dy = _f64(x, w, b, dy)
    C = x.shape[-1]
    n, _, r = _normed(x, groups, eps, stats)
    ww, bb = x.new_ones(C) if w is None else w, x.new_zeros(C) if b is None else b
    flat = n.reshape(x.shape)
    ds = dy * _dsilu(flat * ww + bb) if silu else dy
    dn = (ds * ww).reshape(n.shape)
    mean = lambda t: t.mean((1, 3), keepdim=True)  # noqa: E731
    dx = (r * (dn - mean(dn) - n * mean(dn * n))).reshape(x.shape)
    # (dn is rounded in the activation's slope too: 0.5 of the change of s at most)
    mag = (dy.abs() * (1.1 + 0.5 * (flat * ww).abs() + 0.5 * bb.abs()) if silu else dy.abs())
    dm = (mag * ww.abs()).reshape(n.shape)
    size = (r * (dm * (1 + n.abs()) + mean(dm) + n.abs() * mean(dm * n.abs()))).reshape(x.shape)
    lead = tuple(range(x.dim() - 1))
    got = {"dx": dx, "dw": None if w is None else (ds * flat).sum(lead), "db": None if b is None else ds.sum(lead)}
    sizes = {"dx": size, "dw": (mag * (1 + flat.abs())).sum(lead), "db": mag.sum(lead)}
    return got, sizes
