"""What the gated delta rule operators are measured on: the cases, their inputs, the operators in
plain torch and from their definition in 64 bits.

The operators, per token t and value head h (its key head is h * H_k // H):

  gated delta rule   S_t = e^{g_t} (I - beta_t k_t k_t^T) S_{t-1} + beta_t k_t v_t^T,  o_t = S_t^T q_t
                     over whole sequences ("forward", "packed", "train" with its gradients) and for
                     the tokens of a decode step, S updated in place ("step", "tokens")
  norms before it    q^ = scale q / sqrt(||q||^2 + eps), k^ likewise without the scale,
                     g = -exp(A_log) softplus(a + dt_bias), beta = sigmoid(b)      ("prep")
  norm after it      y = o / sqrt(mean(o^2) + eps) * w * silu(z)                   ("norm")

`own` selects the side that `run` computes: False the plain forms below, True the package's calls.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-6
CHUNK = 64  # of the plain chunked form
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------------ cases
def listed():
    return [
        # a training or prefill batch of the language-model shape
        {"name": "forward_lm", "op": "forward", "B": 8, "T": 2048, "Hk": 16, "H": 16, "dk": 128, "dv": 128,
         "dtype": "bf16", "S0": False},
        # prefill of a packed batch of prompts of uneven lengths, key heads shared by two value heads
        {"name": "forward_packed", "op": "packed", "n": 16, "max_len": 2048, "lens_seed": 5, "Hk": 8, "H": 16,
         "dk": 128, "dv": 128, "dtype": "bf16", "S0": True},
        # a small fp32 model: latency, head size 32
        {"name": "forward_tiny_f32", "op": "forward", "B": 1, "T": 256, "Hk": 2, "H": 2, "dk": 32, "dv": 32,
         "dtype": "f32", "S0": False},
        # one layer of a training step, forward and backward
        {"name": "train_lm", "op": "train", "B": 8, "T": 2048, "Hk": 16, "H": 16, "dk": 128, "dv": 128,
         "dtype": "bf16", "S0": False},
        # the same in fp32, an odd length, shared key heads, from a carried state
        {"name": "train_f32", "op": "train", "B": 2, "T": 300, "Hk": 2, "H": 4, "dk": 64, "dv": 64,
         "dtype": "f32", "S0": True},
        # one token for every sequence of a large serving batch
        {"name": "step_b256", "op": "step", "B": 256, "Hk": 32, "H": 32, "dk": 128, "dv": 128, "dtype": "bf16"},
        # one token for a single user: latency
        {"name": "step_b1", "op": "step", "B": 1, "Hk": 16, "H": 32, "dk": 128, "dv": 128, "dtype": "bf16"},
        # 16 tokens for every sequence: a drafted block, or a continued prompt
        {"name": "tokens_b256m16", "op": "tokens", "B": 256, "m": 16, "Hk": 32, "H": 32, "dk": 128, "dv": 128,
         "dtype": "bf16"},
        # the norms and gates before the mixer in a training step, forward and backward
        {"name": "prep_train", "op": "prep", "B": 8, "T": 2048, "Hk": 16, "H": 16, "dk": 128, "dtype": "bf16",
         "grad": True},
        # the same for one token of a small serving batch: latency
        {"name": "prep_decode", "op": "prep", "B": 16, "T": 1, "Hk": 16, "H": 32, "dk": 128, "dtype": "bf16",
         "grad": False},
        # the gated output norm in a training step, forward and backward
        {"name": "norm_train", "op": "norm", "B": 8, "T": 2048, "H": 16, "dv": 128, "dtype": "bf16", "grad": True},
        # the same for one token of a serving batch
        {"name": "norm_decode", "op": "norm", "B": 256, "T": 1, "H": 32, "dv": 128, "dtype": "bf16", "grad": False},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["forward", "packed", "train", "step", "tokens", "prep", "norm"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    dk = dv = 128
    if rng.random() < 0.5:
        dk = rng.choice([32, 64, 128])
        dv = rng.choice([32, 64, 128])
    Hk = rng.choice([1, 2, 3, 4, 8])
    H = Hk * rng.choice([1, 2, 4])
    c = {"op": op, "dtype": dtype, "H": H}
    if op == "norm":
        c.update(B=_log_int(rng, 1, 8), T=_log_int(rng, 1, 2048), dv=dv, grad=rng.random() < 0.5)
        return c
    c.update(Hk=Hk, dk=dk)
    if op == "prep":
        c.update(B=_log_int(rng, 1, 8), T=_log_int(rng, 1, 2048), grad=rng.random() < 0.5)
        return c
    c.update(dv=dv)
    if op in ("step", "tokens"):
        c.update(B=_log_int(rng, 1, 256))
        if op == "tokens":
            c.update(m=_log_int(rng, 1, 16))
        return c
    c.update(S0=rng.random() < 0.5)
    if op == "packed":
        c.update(n=_log_int(rng, 1, 16), max_len=_log_int(rng, 16, 1024), lens_seed=rng.randrange(1 << 16))
    else:  # at most the token-heads of the language-model shape, a sixteenth of them in fp32
        most = 8 * 2048 * 16 // (1 if dtype == "bf16" else 16)
        B = _log_int(rng, 1, 8)
        c.update(B=B, T=_log_int(rng, 1, max(1, min(4096, most // (B * H)))))
    return c


def _lens(case):
    return np.random.RandomState(case["lens_seed"]).randint(1, case["max_len"] + 1, case["n"]).tolist()


# ------------------------------------------------------------------------------------ inputs
def _unit(x):
    return x / x.norm(dim=-1, keepdim=True)


def prepare(case, seed):
    """Inputs with the distributions of a mixer at work: unit keys, queries of norm 1/sqrt(d_k), one
    decay rate a head (e^g between about 1 and e^-2 a token), step sizes in (0, 1)."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, dt, H = case["op"], DTYPES[case["dtype"]], case["H"]

    def randn(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    def rand(*shape):
        return torch.rand(shape, generator=gen, device="cuda")

    st = {"op": op, "case": case}
    if op == "norm":
        B, T, dv = case["B"], case["T"], case["dv"]
        st.update(o=randn(B, T, H, dv).mul_(0.3).to(dt), z=randn(B, T, H, dv).to(dt), w=1 + 0.1 * randn(dv))
        if case["grad"]:
            st.update(dy=randn(B, T, H, dv).to(dt))
        return st
    Hk, dk = case["Hk"], case["dk"]
    A = 0.5 + 15.5 * rand(H)                              # decay rates
    step = torch.exp(math.log(1e-3) + rand(H) * math.log(1e2))  # typical softplus(a + dt_bias)
    dt_bias = step + torch.log(-torch.expm1(-step))       # its inverse
    if op == "prep":
        B, T = case["B"], case["T"]
        st.update(q=randn(B, T, Hk, dk).to(dt), k=randn(B, T, Hk, dk).to(dt), a=randn(B, T, H).to(dt),
                  b=randn(B, T, H).to(dt), A_log=torch.log(A), dt_bias=dt_bias, scale=dk ** -0.5)
        if case["grad"]:
            st.update(dq=randn(B, T, Hk, dk).to(dt), dk=randn(B, T, Hk, dk).to(dt), dg=randn(B, T, H),
                      dbeta=randn(B, T, H))
        return st
    dv = case["dv"]
    if op == "step":
        lead, rows = (case["B"],), case["B"]
    elif op == "tokens":
        lead, rows = (case["B"], case["m"]), case["B"]
    elif op == "packed":
        lens = _lens(case)
        lead, rows = (1, sum(lens)), len(lens)
        cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
        st.update(lens=lens, cu_seqlens=cu)
    else:
        lead, rows = (case["B"], case["T"]), case["B"]
    st.update(q=_unit(randn(*lead, Hk, dk)).mul_(dk ** -0.5).to(dt),
              k=_unit(randn(*lead, Hk, dk)).to(dt), v=randn(*lead, H, dv).to(dt),
              g=-A * torch.nn.functional.softplus(randn(*lead, H) + dt_bias), beta=torch.sigmoid(randn(*lead, H)))
    if op in ("step", "tokens"):
        st.update(S=0.1 * randn(rows, H, dk, dv))
        return st
    st.update(S0=0.1 * randn(rows, H, dk, dv) if case["S0"] else None)
    if op == "train":
        st.update(dO=randn(*lead, H, dv).to(dt), dS_T=0.1 * randn(rows, H, dk, dv))
    return st


# ------------------------------------------------------------------------------------ the plain forms
def _heads(x, H):
    """[B, T, Hk, d] -> fp32 [B, H, T, d], each key head repeated for its value heads."""
    return x.float().transpose(1, 2).repeat_interleave(H // x.shape[2], dim=1)


def _chunked(q, k, v, g, beta, S):
    """The rule in chunks: q, k, v [B, H, T, d], g, beta [B, H, T], S [B, H, dk, dv] (fp32).  With
    G the running sum of g in a chunk, D_ts = e^{G_t - G_s} (s <= t) and u_t = beta_t (v_t - e^{g_t} S^T k_t):
    (I + tril(beta K K^T o D, -1)) U = beta (V - e^G K S),  O = e^G Q S + (Q K^T o D) U,
    S' = e^{G_C} S + (e^{G_C - G} K)^T U."""
    B, H, T, dv = v.shape
    n = -(-T // CHUNK)
    pad = n * CHUNK - T
    q, k, v = (torch.nn.functional.pad(x, (0, 0, 0, pad)).unflatten(2, (n, CHUNK)) for x in (q, k, v))
    g, beta = (torch.nn.functional.pad(x, (0, pad)).unflatten(2, (n, CHUNK)) for x in (g, beta))
    G = g.double().cumsum(-1)
    low = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=v.device).tril()
    D = (G.unsqueeze(-1) - G.unsqueeze(-2)).masked_fill(~low, -math.inf).exp().float()
    eG, eC, eL = G.exp().float(), (G[..., -1:] - G).exp().float(), G[..., -1].exp().float()
    A = ((k @ k.transpose(-1, -2)) * D * beta.unsqueeze(-1)).tril(-1)
    eye = torch.eye(CHUNK, device=v.device)
    inv, power = eye - A, A @ A  # (I + A)^-1 = (I - A)(I + A^2)(I + A^4) ... as A^64 = 0
    for _ in range(5):
        inv, power = inv + inv @ power, power @ power
    W = inv * beta.unsqueeze(-2)
    U0, WK, P = W @ v, W @ (eG.unsqueeze(-1) * k), (q @ k.transpose(-1, -2)) * D
    qd, kd = eG.unsqueeze(-1) * q, eC.unsqueeze(-1) * k
    out = []
    for c in range(n):
        u = U0[:, :, c] - WK[:, :, c] @ S
        out.append(qd[:, :, c] @ S + P[:, :, c] @ u)
        S = eL[:, :, c, None, None] * S + kd[:, :, c].transpose(-1, -2) @ u
    return torch.stack(out, 2).flatten(2, 3)[:, :, :T], S


def _plain_sequences(st, q, k, v, g, beta, S0):
    H = v.shape[2]
    S = v.new_zeros((v.shape[0], H, q.shape[-1], v.shape[-1]), dtype=torch.float32) if S0 is None else S0
    o, S = _chunked(_heads(q, H), _heads(k, H), _heads(v, H), g.transpose(1, 2), beta.transpose(1, 2), S)
    return o.transpose(1, 2), S


def _plain_packed(st):
    lens, total = st["lens"], st["v"].shape[1]
    n, most = len(lens), max(lens)
    start, length = st["cu_seqlens"][:-1].long(), st["cu_seqlens"].diff().long()
    at = start[:, None] + torch.arange(most, device="cuda")  # [n, most]: token of each padded place
    live = torch.arange(most, device="cuda") < length[:, None]
    at = at.clamp(max=total - 1)
    rows = [st[x][0][at] * live.reshape(n, most, *[1] * (st[x].dim() - 2)) for x in ("q", "k", "v", "g", "beta")]
    o, S = _plain_sequences(st, *rows, st["S0"])
    return o[live].unsqueeze(0).to(st["q"].dtype), S


def _plain_tokens(st, q, k, v, g, beta):
    """q, k [B, m, Hk, dk], v [B, m, H, dv], token by token."""
    H, S, out = v.shape[2], st["S"], []
    q, k, v = (_heads(x, H) for x in (q, k, v))
    new = S
    for t in range(q.shape[2]):
        kt = k[:, :, t].unsqueeze(-1)
        new = g[:, t].exp()[..., None, None] * new
        u = beta[:, t].unsqueeze(-1) * (v[:, :, t] - (new * kt).sum(-2))
        new = new + kt * u.unsqueeze(-2)
        out.append((new * q[:, :, t].unsqueeze(-1)).sum(-2))
    S.copy_(new)
    return torch.stack(out, 1)


def _plain_prep(st):
    def unit(x):
        x = x.float()
        return x * (x.square().sum(-1, keepdim=True) + EPS).rsqrt()

    q, k, a, b = (st[x].float() for x in ("q", "k", "a", "b"))
    t = a + st["dt_bias"]
    sp = t.clamp(min=0) + torch.log1p(torch.exp(-t.abs()))
    rate = torch.exp(st["A_log"])
    beta = 1 / (1 + torch.exp(-b))
    dt = st["q"].dtype
    out = {"q": (unit(q) * st["scale"]).to(dt), "k": unit(k).to(dt), "g": -rate * sp, "beta": beta}
    if "dq" in st:
        def grad(x, dy):
            r = (x.square().sum(-1, keepdim=True) + EPS).rsqrt()
            return r * (dy - x * r * (x * r * dy).sum(-1, keepdim=True))

        da = -st["dg"] * rate / (1 + torch.exp(-t))
        out |= {"dq": (grad(q, st["dq"].float()) * st["scale"]).to(dt), "dk": grad(k, st["dk"].float()).to(dt),
                "da": da.to(dt), "db": (st["dbeta"] * beta * (1 - beta)).to(dt),
                "dA_log": (st["dg"] * out["g"]).double().sum((0, 1)).float(), "ddt_bias": da.double().sum((0, 1)).float()}
    return out


def _plain_norm(st):
    o, z, w = st["o"].float(), st["z"].float(), st["w"]
    r = (o.square().mean(-1, keepdim=True) + EPS).rsqrt()
    s = 1 / (1 + torch.exp(-z))
    n, dt = o * r, st["o"].dtype
    out = {"y": (n * w * z * s).to(dt)}
    if "dy" in st:
        dy = st["dy"].float()
        dn = dy * w * z * s
        out |= {"do": (r * (dn - n * (dn * n).mean(-1, keepdim=True))).to(dt),
                "dz": (dy * n * w * s * (1 + z * (1 - s))).to(dt),
                "dw": (dy * n * z * s).double().sum((0, 1, 2)).float()}
    return out


def _plain(st):
    op = st["op"]
    if op == "prep":
        return _plain_prep(st)
    if op == "norm":
        return _plain_norm(st)
    dt = st["q"].dtype
    if op == "step":
        o = _plain_tokens(st, *(st[x].unsqueeze(1) for x in ("q", "k", "v", "g", "beta")))
        return {"o": o.squeeze(1).to(dt), "S": st["S"]}
    args = [st[x] for x in ("q", "k", "v", "g", "beta")]
    if op == "tokens":
        return {"o": _plain_tokens(st, *args).to(dt), "S": st["S"]}
    if op == "packed":
        o, S = _plain_packed(st)
        return {"o": o, "S_T": S}
    if op == "forward":
        o, S = _plain_sequences(st, *args, st["S0"])
        return {"o": o.to(dt), "S_T": S}
    B, _, H, dv = st["v"].shape
    S0 = torch.zeros(B, H, st["q"].shape[-1], dv, device="cuda") if st["S0"] is None else st["S0"]
    leaves = [x.float().detach().requires_grad_() for x in (*args, S0)]
    with torch.enable_grad():
        o, S = _plain_sequences(st, *leaves)
        grads = torch.autograd.grad([o, S], leaves, [st["dO"].float(), st["dS_T"]])
    out = {"o": o.detach().to(dt), "S_T": S.detach()}
    for name, x in zip(("dq", "dk", "dv", "dg", "dbeta", "dS0"), grads):
        out[name] = x.to(dt) if name in ("dq", "dk", "dv") else x
    return out


# ------------------------------------------------------------------------------------ the package's calls
def _own(st):
    import exact_delta_rule_gb300 as efla

    op = st["op"]
    if op == "prep":
        args = (st["q"], st["k"], st["a"], st["b"], st["A_log"], st["dt_bias"])
        out = efla.gated_prep(*args, scale=st["scale"], eps=EPS)
        if "dq" in st:
            out = {**out, **efla.gated_prep_bwd(*args, st["dq"], st["dk"], st["dg"], st["dbeta"], scale=st["scale"],
                                                eps=EPS)}
        return out
    if op == "norm":
        out = {"y": efla.norm_gate(st["o"], st["z"], st["w"], eps=EPS)}
        if "dy" in st:
            out |= efla.norm_gate_bwd(st["o"], st["z"], st["w"], st["dy"], eps=EPS)
        return out
    args = (st["q"], st["k"], st["v"], st["g"], st["beta"])
    if op == "step":
        return {"o": efla.gated_decode_step(*args, st["S"]), "S": st["S"]}
    if op == "tokens":
        return {"o": efla.gated_decode_tokens(*args, st["S"]), "S": st["S"]}
    if op == "packed":
        o, S = efla.gated_fwd_chunked(*args, st["S0"], st["cu_seqlens"])
        return {"o": o, "S_T": S}
    if op == "forward":
        o, S = efla.gated_fwd_chunked(*args, st["S0"])
        return {"o": o, "S_T": S}
    o, S, ws = efla.gated_fwd_chunked_train(*args, st["S0"])
    grads = efla.gated_bwd_chunked(*args, st["S0"], st["dO"], st["dS_T"], workspace=ws, saved=True)
    return {"o": o, "S_T": S, **{x: grads[x] for x in ("dq", "dk", "dv", "dg", "dbeta", "dS0")}}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------------------------ what it cannot do without
def work(case):
    op, H, es = case["op"], case["H"], 2 if case["dtype"] == "bf16" else 4
    if op == "norm":
        n = case["B"] * case["T"] * H * case["dv"]
        return {"bytes": n * es * (6 if case["grad"] else 3), "flops": n * (24 if case["grad"] else 9)}
    Hk, dk = case["Hk"], case["dk"]
    if op == "prep":
        tok = case["B"] * case["T"]
        vec, gate = 2 * tok * Hk * dk * es, tok * H  # q and k
        b = 2 * vec + gate * (2 * es + 8)
        f = 4 * tok * Hk * dk * 2 + gate * 12
        if case["grad"]:
            b, f = b + 2 * vec + gate * (2 * es + 8), f + 8 * tok * Hk * dk * 2 + gate * 20
        return {"bytes": b, "flops": f}
    dv = case["dv"]
    if op == "step":
        tok, units = case["B"], case["B"] * H
    elif op == "tokens":
        tok, units = case["B"] * case["m"], case["B"] * H
    elif op == "packed":
        tok, units = sum(_lens(case)), case["n"] * H
    else:
        tok, units = case["B"] * case["T"], case["B"] * H
    io = tok * (2 * Hk * dk * es + 2 * H * dv * es + 8 * H)  # q, k, v, o, g, beta
    state = units * dk * dv * 4
    if op in ("step", "tokens"):
        return {"bytes": io + 2 * state, "flops": tok * H * 6 * dk * dv}
    C = CHUNK
    fwd = tok * H * (6 * dk * dv + 3 * C * dk + 2 * C * dv + C * C / 3)
    if op != "train":
        return {"bytes": io + state * (2 if case["S0"] else 1), "flops": fwd}
    io += tok * (2 * Hk * dk * es + 2 * H * dv * es + 8 * H)  # dq, dk, dv, dO, dg, dbeta
    bwd = tok * H * (12 * dk * dv + 3 * C * dk + 4 * C * dv)
    return {"bytes": io + state * (4 if case["S0"] else 3), "flops": fwd + bwd}


# ------------------------------------------------------------------------------------ 64 bits, by the definition
def _exact_scan(q, k, v, g, beta, S, keep):
    """One token after the other in 64 bits on [B, T, H, d]; with `keep` also what each token started from."""
    outs, kept = [], []
    for t in range(q.shape[1]):
        if keep:
            kept.append(S)
        Sd = S * g[:, t].exp()[..., None, None]
        u = beta[:, t, :, None] * (v[:, t] - torch.einsum("bhkv,bhk->bhv", Sd, k[:, t]))
        S = Sd + k[:, t, :, :, None] * u[:, :, None, :]
        outs.append(torch.einsum("bhkv,bhk->bhv", S, q[:, t]))
    return torch.stack(outs, 1), S, kept


def _exact_reverse(q, k, v, g, beta, kept, dO, dS):
    """Reverse mode of the same, last token first."""
    r = {x: [] for x in ("dq", "dk", "dv", "dg", "dbeta")}
    for t in reversed(range(q.shape[1])):
        kt, qt, bt, S = k[:, t], q[:, t], beta[:, t, :, None], kept[t]
        Sd = S * g[:, t].exp()[..., None, None]
        e = v[:, t] - torch.einsum("bhkv,bhk->bhv", Sd, kt)
        u = bt * e
        new = Sd + kt[..., None] * u[:, :, None]
        r["dq"].append(torch.einsum("bhkv,bhv->bhk", new, dO[:, t]))
        dS = dS + qt[..., None] * dO[:, t, :, None]
        du = torch.einsum("bhkv,bhk->bhv", dS, kt)
        de = bt * du
        r["dk"].append(torch.einsum("bhkv,bhv->bhk", dS, u) - torch.einsum("bhkv,bhv->bhk", Sd, de))
        r["dv"].append(de)
        r["dbeta"].append((du * e).sum(-1))
        dSd = dS - kt[..., None] * de[:, :, None]
        r["dg"].append((dSd * Sd).sum((-1, -2)))
        dS = dSd * g[:, t].exp()[..., None, None]
    return {x: torch.stack(y[::-1], 1) for x, y in r.items()} | {"dS0": dS}


def exact(case, seed):
    st = prepare(case, seed)
    op, d = st["op"], {x: y.double() for x, y in st.items() if torch.is_tensor(y) and y.is_floating_point()}
    if op == "norm":
        o, z, w = d["o"], d["z"], d["w"]
        rms = (o.pow(2).sum(-1, keepdim=True) / o.shape[-1] + EPS).sqrt()
        gate = z * torch.sigmoid(z)
        out = {"y": o / rms * w * gate}
        if case["grad"]:
            dn = d["dy"] * w * gate
            out["do"] = dn / rms - o * (dn * o).sum(-1, keepdim=True) / (o.shape[-1] * rms ** 3)
            out["dz"] = d["dy"] * o / rms * w * (torch.sigmoid(z) + gate * (1 - torch.sigmoid(z)))
            out["dw"] = (d["dy"] * o / rms * gate).flatten(0, 2).sum(0)
        return out
    if op == "prep":
        nq, nk = ((d[x].pow(2).sum(-1, keepdim=True) + EPS).sqrt() for x in ("q", "k"))
        x, sig = d["a"] + d["dt_bias"], torch.sigmoid(d["b"])
        g = -d["A_log"].exp() * torch.nn.functional.softplus(x)
        out = {"q": st["scale"] * d["q"] / nq, "k": d["k"] / nk, "g": g, "beta": sig}
        if case["grad"]:
            out["dq"] = st["scale"] * (d["dq"] / nq - d["q"] * (d["q"] * d["dq"]).sum(-1, keepdim=True) / nq ** 3)
            out["dk"] = d["dk"] / nk - d["k"] * (d["k"] * d["dk"]).sum(-1, keepdim=True) / nk ** 3
            out["da"] = -d["dg"] * d["A_log"].exp() * torch.sigmoid(x)
            out["db"] = d["dbeta"] * sig * torch.sigmoid(-d["b"])
            out["dA_log"], out["ddt_bias"] = (d["dg"] * g).sum((0, 1)), out["da"].sum((0, 1))
        return out
    H = case["H"]
    if op == "step":
        for x in ("q", "k", "v", "g", "beta"):
            d[x] = d[x].unsqueeze(1)
    rep = H // case["Hk"]
    q, k = (d[x].repeat_interleave(rep, 2) for x in ("q", "k"))
    v, g, beta = d["v"], d["g"], d["beta"]
    if op in ("step", "tokens"):
        o, S, _ = _exact_scan(q, k, v, g, beta, d["S"], False)
        return {"o": o[:, 0] if op == "step" else o, "S": S}
    B = v.shape[0]
    if op == "packed":
        outs, states, at = [], [], 0
        for i, n in enumerate(st["lens"]):
            S = d["S0"][i:i + 1] if case["S0"] else v.new_zeros(1, H, case["dk"], case["dv"])
            s = slice(at, at + n)
            o, S, _ = _exact_scan(q[:, s], k[:, s], v[:, s], g[:, s], beta[:, s], S, False)
            outs.append(o)
            states.append(S)
            at += n
        return {"o": torch.cat(outs, 1), "S_T": torch.cat(states)}
    S0 = d["S0"] if case["S0"] else v.new_zeros(B, H, case["dk"], case["dv"])
    o, S, kept = _exact_scan(q, k, v, g, beta, S0, op == "train")
    out = {"o": o, "S_T": S}
    if op == "train":
        out |= _exact_reverse(q, k, v, g, beta, kept, d["dO"], d["dS_T"])
        for x in ("dq", "dk"):
            out[x] = out[x].unflatten(2, (case["Hk"], rep)).sum(3)
    return out
