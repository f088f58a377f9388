"""Gated delta rule and the norms around it in 64 bits, straight from the definitions (torch, any
device): the token recurrence, its reverse mode written out by hand, and the row norms.

    S_t = e^{g_t} (I - alpha_t k_t k_t^T) S_{t-1} + alpha_t k_t v_t^T,   o_t = S_t^T q_t

q, k [B, T, Hk, dk], v [B, T, H, dv], g, beta [B, T, H]; value head h reads key head h // (H // Hk).
alpha = beta ("euler") or (1 - e^{-beta lambda}) / lambda with lambda = ||k||^2 ("exact", beta at 0).
"""
from __future__ import annotations

import torch


def _f64(*xs):
    return [None if x is None else x.detach().double() for x in xs]


def _gate(beta, lam, update):
    """alpha, d alpha / d beta, d alpha / d lambda."""
    if update == "euler":
        return beta, torch.ones_like(beta), torch.zeros_like(beta)
    z = beta * lam
    safe = torch.where(lam > 0, lam, torch.ones_like(lam))
    alpha = torch.where(lam > 0, -torch.expm1(-z) / safe, beta)
    # d alpha / d lambda = (beta e^{-z} - alpha) / lambda, by its series in z where that cancels
    series, term = torch.zeros_like(z), torch.full_like(z, 0.5)
    for n in range(2, 30):  # beta^2 sum_n (-1)^{n-1} (n-1) z^{n-2} / n!
        series = series + (-1) ** (n - 1) * (n - 1) * term
        term = term * z / (n + 1)
    dl = torch.where(z.abs() > 1, (beta * torch.exp(-z) - alpha) / safe, beta * beta * series)
    return alpha, torch.exp(-z), dl


def fwd(q, k, v, g, beta, S0=None, update="euler", keep=False):
    """(o, S_T) [and, with `keep`, the state every token starts from]."""
    q, k, v, g, beta, S0 = _f64(q, k, v, g, beta, S0)
    B, T, H, dv = v.shape
    rep = H // q.shape[2]
    q, k = q.repeat_interleave(rep, 2), k.repeat_interleave(rep, 2)
    S = v.new_zeros(B, H, q.shape[-1], dv) if S0 is None else S0
    o, kept = v.new_zeros(B, T, H, dv), []
    for t in range(T):
        kept.append(S)
        kt = k[:, t]
        alpha = _gate(beta[:, t], (kt * kt).sum(-1), update)[0]
        Sd = g[:, t].exp()[..., None, None] * S
        u = alpha[..., None] * (v[:, t] - (Sd * kt[..., None]).sum(-2))
        S = Sd + kt[..., None] * u[..., None, :]
        o[:, t] = (S * q[:, t][..., None]).sum(-2)
    return (o, S, kept) if keep else (o, S)


def bwd(q, k, v, g, beta, S0, dO, dS_T=None, update="euler"):
    """Gradients of any loss with dL/do = dO and dL/dS_T = dS_T."""
    _, S_T, kept = fwd(q, k, v, g, beta, S0, update, keep=True)
    q, k, v, g, beta, dO, dS_T = _f64(q, k, v, g, beta, dO, dS_T)
    B, T, H, dv = v.shape
    Hk, dk = q.shape[2:]
    rep = H // Hk
    qh, kh = q.repeat_interleave(rep, 2), k.repeat_interleave(rep, 2)
    G = torch.zeros_like(S_T) if dS_T is None else dS_T
    dq, dk_, dv_ = torch.zeros_like(qh), torch.zeros_like(kh), torch.zeros_like(v)
    dg, dbeta = torch.zeros_like(g), torch.zeros_like(beta)
    for t in range(T - 1, -1, -1):
        kt, qt, S = kh[:, t], qh[:, t], kept[t]
        alpha, dadb, dadl = _gate(beta[:, t], (kt * kt).sum(-1), update)
        decay = g[:, t].exp()[..., None, None]
        Sd = decay * S
        e = v[:, t] - (Sd * kt[..., None]).sum(-2)
        u = alpha[..., None] * e
        new = Sd + kt[..., None] * u[..., None, :]
        dq[:, t] = (new * dO[:, t][..., None, :]).sum(-1)
        G = G + qt[..., None] * dO[:, t][..., None, :]
        du = (G * kt[..., None]).sum(-2)
        de = alpha[..., None] * du
        dalpha = (du * e).sum(-1)
        dk_[:, t] = (G * u[..., None, :]).sum(-1) - (Sd * de[..., None, :]).sum(-1) + (2 * dalpha * dadl)[..., None] * kt
        dv_[:, t] = de
        dbeta[:, t] = dalpha * dadb
        G = G - kt[..., None] * de[..., None, :]
        dg[:, t] = (G * Sd).sum((-1, -2))
        G = decay * G
    fold = lambda x: x.reshape(B, T, Hk, rep, dk).sum(3)  # noqa: E731
    return {"dq": fold(dq), "dk": fold(dk_), "dv": dv_, "dg": dg, "dbeta": dbeta, "dS0": G}


def prep(q, k, a, b, A_log, dt_bias, scale=1.0, eps=1e-6):
    q, k, a, b, A_log, dt_bias = _f64(q, k, a, b, A_log, dt_bias)
    unit = lambda x: x / torch.sqrt((x * x).sum(-1, keepdim=True) + eps)  # noqa: E731
    x = a + dt_bias
    softplus = torch.maximum(x, torch.zeros_like(x)) + torch.log1p(torch.exp(-x.abs()))
    return {"q": scale * unit(q), "k": unit(k), "g": -torch.exp(A_log) * softplus, "beta": 1 / (1 + torch.exp(-b))}


def prep_bwd(q, k, a, b, A_log, dt_bias, dq, dk, dg, dbeta, scale=1.0, eps=1e-6):
    out = prep(q, k, a, b, A_log, dt_bias, scale, eps)
    q, k, a, b, dq, dk, dg, dbeta, A_log, dt_bias = _f64(q, k, a, b, dq, dk, dg, dbeta, A_log, dt_bias)

    def grad(x, dy):
        n = torch.sqrt((x * x).sum(-1, keepdim=True) + eps)
        return dy / n - x * (x * dy).sum(-1, keepdim=True) / n ** 3

    da = -dg * torch.exp(A_log) / (1 + torch.exp(-(a + dt_bias)))
    lead = tuple(range(a.dim() - 1))
    return {"dq": scale * grad(q, dq), "dk": grad(k, dk), "da": da, "db": dbeta * out["beta"] / (1 + torch.exp(b)),
            "dA_log": (dg * out["g"]).sum(lead), "ddt_bias": da.sum(lead)}


def norm_gate(o, z, w, eps=1e-6):
    o, z, w = _f64(o, z, w)
    return o / torch.sqrt((o * o).mean(-1, keepdim=True) + eps) * w * z / (1 + torch.exp(-z))


def norm_gate_bwd(o, z, w, dy, eps=1e-6):
    o, z, w, dy = _f64(o, z, w, dy)
    rms = torch.sqrt((o * o).mean(-1, keepdim=True) + eps)
    s = 1 / (1 + torch.exp(-z))
    dn = dy * w * z * s
    return {"do": dn / rms - o * (dn * o).mean(-1, keepdim=True) / rms ** 3,
            "dz": dy * o / rms * w * (s + z * s * (1 - s)),
            "dw": (dy * o / rms * z * s).flatten(0, -2).sum(0)}
