"""What the selective state space scan, its short causal convolution and the group norm are measured on: the
cases, their inputs, the operators in plain torch and from their definition in 64 bits.

Per token t and channel d (of D; B and C are shared by the D / G channels of a group, channel d reads group
d * G // D):

  short convolution  s_t = bias + sum_{j < W} w_j x_{t-W+1+j},  y = s or silu(s), the W - 1 inputs before a
                     sequence from its state; over whole sequences ("conv", "conv_packed", "conv_train" with its
                     gradients) and for one token, state in place ("conv_step")
  selective scan     delta_t = softplus(dt_t + dt_bias),  h_t = exp(-exp(A_log) delta_t) h_{t-1} + delta_t x_t B_t,
                     y_t = (C_t . h_t + D x_t) silu(z_t), h of N entries a channel; "scan", "scan_packed",
                     "scan_train" with its gradients, "scan_step" for one token, state in place
  group norm         n = (x - mean) / sqrt(var + eps) over the L positions and C / groups channels of a group,
                     y = w n + b or silu of it, channels last ("norm")

`own` selects the side that `run` computes: False the plain forms below, True the package's calls.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-5
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------------ cases
def listed():
    return [
        # the convolution before a mixer in a training or prefill batch: q, k and v of 16 heads of 128
        {"name": "conv_prompt", "op": "conv", "B": 8, "T": 2048, "D": 6144, "W": 4, "dtype": "bf16", "act": "silu",
         "bias": True, "S0": False},
        # one layer's convolution in a training step, forward and backward
        {"name": "conv_train", "op": "conv_train", "B": 8, "T": 2048, "D": 2048, "W": 4, "dtype": "bf16", "act": "silu",
         "bias": True, "S0": False},
        # one token for every sequence of a large serving batch
        {"name": "conv_step_b256", "op": "conv_step", "B": 256, "D": 6144, "W": 4, "dtype": "bf16", "act": "silu",
         "bias": True},
        # a training or prefill batch
        {"name": "scan_prompt", "op": "scan", "B": 8, "T": 2048, "D": 4096, "N": 16, "G": 1, "dtype": "bf16", "z": True,
         "S0": False},
        # prefill of a packed batch of prompts of uneven lengths, continued from their states
        {"name": "scan_packed", "op": "scan_packed", "n": 16, "max_len": 2048, "lens_seed": 5, "D": 2048, "N": 16, "G": 1,
         "dtype": "bf16", "z": True, "S0": True},
        # one long prompt of a single user
        {"name": "scan_long", "op": "scan", "B": 1, "T": 12001, "D": 2048, "N": 16, "G": 1, "dtype": "bf16", "z": True,
         "S0": False},
        # one layer of a training step, forward and backward
        {"name": "scan_train", "op": "scan_train", "B": 8, "T": 2048, "D": 2048, "N": 16, "G": 1, "dtype": "bf16",
         "z": True, "S0": False},
        # the same of a small fp32 model: odd lengths, a larger state, two groups, from a carried state
        {"name": "scan_train_f32", "op": "scan_train", "B": 2, "T": 301, "D": 520, "N": 64, "G": 2, "dtype": "f32",
         "z": True, "S0": True},
        # one token for every sequence of a large serving batch
        {"name": "scan_step_b256", "op": "scan_step", "B": 256, "D": 4096, "N": 16, "G": 1, "dtype": "bf16", "z": True},
        # one token for a single user: latency
        {"name": "scan_step_b1", "op": "scan_step", "B": 1, "D": 2048, "N": 16, "G": 1, "dtype": "bf16", "z": True},
        # the norm of a mixer's 16 heads of 128, token by token, in a training step, forward and backward
        {"name": "norm_heads_train", "op": "norm", "rows": 16384, "L": 1, "C": 2048, "groups": 16, "dtype": "bf16",
         "act": None, "grad": True},
        # feature maps of 64 x 64 positions in groups of 10 channels
        {"name": "norm_map", "op": "norm", "rows": 8, "L": 4096, "C": 320, "groups": 32, "dtype": "bf16", "act": "silu",
         "grad": False},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case of the same ranges: bf16 and fp32, one token to thousands, channels in steps of 8."""
    op = rng.choice(["conv", "conv_packed", "conv_train", "conv_step", "scan", "scan_packed", "scan_train", "scan_step",
                     "norm", "norm"])
    c = {"op": op, "dtype": rng.choice(["bf16", "bf16", "f32"])}
    if op == "norm":
        groups, each = rng.choice([1, 2, 3, 4, 8, 16, 32]), _log_int(rng, 1, 256)
        C = -(-groups * each // 8) * 8
        while C % groups:
            C += 8
        L = 1 if rng.random() < 0.4 else _log_int(rng, 2, 4096)
        c.update(L=L, C=C, groups=groups, rows=_log_int(rng, 1, max(1, min(16384, (1 << 23) // (L * C)))),
                 act=rng.choice([None, "silu"]), grad=rng.random() < 0.5)
        return c
    D = 8 * _log_int(rng, 1, 512)
    if op.startswith("conv"):
        c.update(W=rng.choice([2, 3, 4, 4]), act=rng.choice([None, "silu", "silu"]), bias=rng.random() < 0.7)
    else:
        N = rng.choice([16, 16, 32, 64, 128])
        G = rng.choice([1, 1, 2, 4])
        D = -(-D // (8 * G)) * 8 * G
        c.update(N=N, G=G, z=rng.random() < 0.7)
    c.update(D=D)
    if op.endswith("step"):
        c.update(B=_log_int(rng, 1, 256))
        if op == "scan_step":
            c["B"] = max(1, min(c["B"], 256 * 4096 * 16 // (D * c["N"])))
        return c
    c.update(S0=rng.random() < 0.5)
    most = 8 * 2048 * 2048 // D if op.startswith("conv") else 8 * 2048 * 2048 * 16 // (D * c["N"])
    if op.endswith("packed"):
        n = _log_int(rng, 1, 16)
        c.update(n=n, max_len=_log_int(rng, 1, max(1, min(2048, most // n))), lens_seed=rng.randrange(1 << 16))
    else:
        B = _log_int(rng, 1, 8)
        c.update(B=B, T=_log_int(rng, 1, max(1, min(4096, most // B))))
    return c


def _lens(case):
    return np.random.RandomState(case["lens_seed"]).randint(1, case["max_len"] + 1, case["n"]).tolist()


# ------------------------------------------------------------------------------------ inputs
def prepare(case, seed):
    """Inputs with the distributions of a mixer at work: step sizes softplus(dt + dt_bias) around a rate between
    1e-3 and 1e-1 a channel, decay rates 1 .. N, convolution weights of a default initialisation, activations of
    order one."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, dt = case["op"], DTYPES[case["dtype"]]

    def randn(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    def rand(*shape):
        return torch.rand(shape, generator=gen, device="cuda")

    st = {"op": op, "case": case}
    if op == "norm":
        rows, L, C = case["rows"], case["L"], case["C"]
        st.update(x=(randn(rows, L, C) * (0.5 + rand(C)) + 0.5 * randn(C)).to(dt), w=1 + 0.1 * randn(C), b=0.1 * randn(C))
        if case["grad"]:
            st.update(dy=randn(rows, L, C).to(dt))
        return st
    D = case["D"]
    if op.endswith("step"):
        lead, rows = (case["B"],), case["B"]
    elif op.endswith("packed"):
        lens = _lens(case)
        lead, rows = (1, sum(lens)), len(lens)
        cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
        st.update(lens=lens, cu_seqlens=cu)
    else:
        lead, rows = (case["B"], case["T"]), case["B"]
    st.update(x=randn(*lead, D).to(dt))
    if op.startswith("conv"):
        W = case["W"]
        st.update(w=(2 * rand(D, W) - 1) * W ** -0.5, bias=(2 * rand(D) - 1) * W ** -0.5 if case["bias"] else None)
        state = randn(rows, W - 1, D).to(dt)
        if op == "conv_train":
            st.update(dy=randn(*lead, D).to(dt), dstate_T=randn(rows, W - 1, D).to(dt))
    else:
        N, G = case["N"], case["G"]
        step = torch.exp(math.log(1e-3) + rand(D) * math.log(1e2))
        st.update(dt=(0.5 * randn(*lead, D)).to(dt), dt_bias=step + torch.log(-torch.expm1(-step)),
                  A_log=torch.log(torch.arange(1, N + 1, device="cuda").float()).expand(D, N) + 0.05 * randn(D, N),
                  Bm=randn(*lead, G, N).to(dt), Cm=randn(*lead, G, N).to(dt), D=1 + 0.1 * randn(D),
                  z=randn(*lead, D).to(dt) if case["z"] else None)
        state = 0.3 * randn(rows, D, N)
        if op == "scan_train":
            st.update(dy=randn(*lead, D).to(dt), dS_T=0.1 * randn(rows, D, N))
    if op.endswith("step"):
        st.update(state=state)
    else:
        st.update(state0=state if case["S0"] else None)
    return st


# ------------------------------------------------------------------------------------ the plain forms
def _silu(s):
    return s / (1 + torch.exp(-s))


def _dsilu(s):
    g = 1 / (1 + torch.exp(-s))
    return g * (1 + s * (1 - g))


def _softplus(t):
    return t.clamp(min=0) + torch.log1p(torch.exp(-t.abs()))


def _history(st):
    """x behind the W - 1 inputs that its sequences continue, fp32 [B, W - 1 + T, D]."""
    x, W = st["x"].float(), st["w"].shape[1]
    before = x.new_zeros(x.shape[0], W - 1, x.shape[2]) if st["state0"] is None else st["state0"].float()
    return torch.cat([before, x], 1)


def _plain_conv(st):
    case, w = st["case"], st["w"]
    W, dt = case["W"], st["x"].dtype
    if st["op"] == "conv_step":
        x = torch.cat([st["state"].float(), st["x"].float().unsqueeze(1)], 1)
        s = sum(w[:, j] * x[:, j] for j in range(W))
    elif st["op"] == "conv_packed":
        x, cu = st["x"].float(), st["cu_seqlens"].long()
        T, n = x.shape[1], len(st["lens"])
        seq = torch.repeat_interleave(torch.arange(n, device="cuda"), cu.diff(), output_size=T)
        at = torch.arange(T, device="cuda") - cu[seq]  # a token's place in its sequence
        zero = x.new_zeros(n, W - 1, case["D"])
        before = zero if st["state0"] is None else st["state0"].float()
        taps = []
        for j in range(W):
            back = W - 1 - j
            old = before[seq, (at - back + W - 1).clamp(0, W - 2)]
            taps.append(torch.where((at >= back)[:, None], x[0].roll(back, 0), old))
        s = sum(w[:, j] * taps[j] for j in range(W)).unsqueeze(0)
        place = cu[1:, None] - (W - 1) + torch.arange(W - 1, device="cuda")  # the last W - 1 inputs
        inside = place >= cu[:-1, None]
        old = before.gather(1, (place - cu[:-1, None] + W - 1).clamp(0, W - 2)[..., None].expand_as(before))
        state = torch.where(inside[..., None], x[0][place.clamp(min=0)], old).to(dt)
    else:
        x = _history(st)
        T = st["x"].shape[1]
        s = sum(w[:, j] * x[:, j:j + T] for j in range(W))
        state = x[:, T:].to(dt)
    if st["bias"] is not None:
        s = s + st["bias"]
    y = (_silu(s) if case["act"] else s).to(dt)
    if st["op"] == "conv_step":
        st["state"].copy_(x[:, 1:])
        return {"y": y, "state": st["state"]}
    out = {"y": y, "state_T": state}
    if st["op"] == "conv_train":
        ds = st["dy"].float()
        if case["act"]:
            ds = ds * _dsilu(s)
        dx = torch.zeros_like(x)
        for j in range(W):
            dx[:, j:j + T] += w[:, j] * ds
        dx[:, T:] += st["dstate_T"].float()
        out["dx"], out["dstate0"] = dx[:, W - 1:].to(dt), dx[:, :W - 1].to(dt)
        out["dw"] = torch.stack([(ds * x[:, j:j + T]).double().sum((0, 1)) for j in range(W)], 1).float()
        if st["bias"] is not None:
            out["dbias"] = ds.double().sum((0, 1)).float()
    return out


def _plain_scan(st, x, dt, Bm, Cm, z, h):
    """Token by token over [B, T, ...]: (y in fp32, the last state, the state that each token starts from)."""
    case = st["case"]
    rate, rep = -torch.exp(st["A_log"]), case["D"] // case["G"]
    delta = _softplus(dt.float() + st["dt_bias"])
    if "live" in st:
        delta = delta * st["live"]
    x = x.float()
    B, T, D = x.shape
    u, ys, kept = delta * x, torch.empty_like(x), []
    keep = st["op"] == "scan_train"
    for t in range(T):
        if keep:
            kept.append(h)
        b, c = (m[:, t].float().repeat_interleave(rep, 1) if case["G"] > 1 else m[:, t].float() for m in (Bm, Cm))
        h = torch.exp(delta[:, t, :, None] * rate) * h + u[:, t, :, None] * b
        ys[:, t] = (h * c).sum(-1)
    out = ys + st["D"] * x
    return (out if z is None else out * _silu(z.float())), h, (ys, delta, kept)


def _plain_scan_grads(st, ys, delta, kept):
    case = st["case"]
    D, N, G = case["D"], case["N"], case["G"]
    rate, rep = -torch.exp(st["A_log"]), D // G
    x, Bm, Cm, dy = (st[k].float() for k in ("x", "Bm", "Cm", "dy"))
    B, T, _ = x.shape
    out = {}
    if st["z"] is not None:
        z = st["z"].float()
        out["dz"] = dy * (ys + st["D"] * x) * _dsilu(z)
        dy = dy * _silu(z)
    du, ddelta, dB, dC = (torch.empty_like(m) for m in (x, x, Bm, Cm))
    drate = torch.zeros(B, D, N, device="cuda", dtype=torch.float64)
    dh, u = st["dS_T"], delta * x
    for t in reversed(range(T)):
        b, c = (m[:, t].repeat_interleave(rep, 1) if G > 1 else m[:, t] for m in (Bm, Cm))
        a = torch.exp(delta[:, t, :, None] * rate)
        h = a * kept[t] + u[:, t, :, None] * b
        dh = dh + dy[:, t, :, None] * c
        dC[:, t] = (h * dy[:, t, :, None]).unflatten(1, (G, rep)).sum(2)
        dB[:, t] = (dh * u[:, t, :, None]).unflatten(1, (G, rep)).sum(2)
        du[:, t] = (dh * b).sum(-1)
        dh = dh * a
        w = dh * kept[t]
        ddelta[:, t] = (w * rate).sum(-1)
        drate += w * delta[:, t, :, None]
    ddelta = ddelta + du * x
    ddt = ddelta / (1 + torch.exp(-(st["dt"].float() + st["dt_bias"])))
    out |= {"dx": du * delta + st["D"] * dy, "ddt": ddt, "dB": dB, "dC": dC}
    out = {k: v.to(st["x"].dtype) for k, v in out.items()}
    out["dA_log"] = (drate.sum(0) * rate).float()
    out["dD"] = (dy * x).double().sum((0, 1)).float()
    out["ddt_bias"] = ddt.double().sum((0, 1)).float()
    out["dS0"] = dh
    return out


def _plain_ssm(st):
    op, case, dt = st["op"], st["case"], st["x"].dtype
    args = [st[k] for k in ("x", "dt", "Bm", "Cm", "z")]
    if op == "scan_step":
        y, h, _ = _plain_scan(st, *(None if a is None else a.unsqueeze(1) for a in args), st["state"])
        st["state"].copy_(h)
        return {"y": y.squeeze(1).to(dt), "S": st["state"]}
    rows = len(st["lens"]) if op == "scan_packed" else case["B"]
    h = torch.zeros(rows, case["D"], case["N"], device="cuda") if st["state0"] is None else st["state0"]
    if op == "scan_packed":  # rows of the longest length; a place past its sequence's end has a step of 0
        lens, total = st["lens"], st["x"].shape[1]
        most = max(lens)
        start, length = st["cu_seqlens"][:-1].long(), st["cu_seqlens"].diff().long()
        at = start[:, None] + torch.arange(most, device="cuda")
        live = torch.arange(most, device="cuda") < length[:, None]
        at = at.clamp(max=total - 1)
        y, h, _ = _plain_scan(st | {"live": live[..., None].float()}, *(None if a is None else a[0][at] for a in args), h)
        return {"y": y[live].unsqueeze(0).to(dt), "S_T": h}
    y, h, rest = _plain_scan(st, *args, h)
    out = {"y": y.to(dt), "S_T": h}
    return out | _plain_scan_grads(st, *rest) if op == "scan_train" else out


def _plain_norm(st):
    case, x, w, b = st["case"], st["x"].float(), st["w"], st["b"]
    rows, L, C = x.shape
    xg = x.unflatten(2, (case["groups"], -1))
    mean = xg.mean((1, 3), keepdim=True)
    r = 1 / (((xg - mean).square()).mean((1, 3), keepdim=True) + EPS).sqrt()
    n = ((xg - mean) * r).flatten(2)
    s, dt = n * w + b, st["x"].dtype
    out = {"y": (_silu(s) if case["act"] else s).to(dt)}
    if case["grad"]:
        ds = st["dy"].float()
        if case["act"]:
            ds = ds * _dsilu(s)
        dn, ng = (ds * w).unflatten(2, (case["groups"], -1)), n.unflatten(2, (case["groups"], -1))
        dx = r * (dn - dn.mean((1, 3), keepdim=True) - ng * (dn * ng).mean((1, 3), keepdim=True))
        out["dx"] = dx.flatten(2).to(dt)
        out["dw"], out["db"] = (ds * n).double().sum((0, 1)).float(), ds.double().sum((0, 1)).float()
    return out


def _plain(st):
    op = st["op"]
    return _plain_norm(st) if op == "norm" else _plain_conv(st) if op.startswith("conv") else _plain_ssm(st)


# ------------------------------------------------------------------------------------ the package's calls
def _own(st):
    import exact_delta_rule_gb300 as efla

    op, act = st["op"], st["case"].get("act")
    if op == "norm":
        args = (st["x"], st["w"], st["b"], st["case"]["groups"])
        if not st["case"]["grad"]:
            return {"y": efla.group_norm(*args, eps=EPS, activation=act)}
        y, stats = efla.group_norm(*args, eps=EPS, activation=act, return_stats=True)
        return {"y": y, **efla.group_norm_bwd(*args, stats, st["dy"], activation=act)}
    if op.startswith("conv"):
        args = (st["x"], st["w"], st["bias"])
        if op == "conv_step":
            return {"y": efla.causal_conv_step(*args, st["state"], activation=act), "state": st["state"]}
        y, state = efla.causal_conv(*args, st["state0"], st.get("cu_seqlens"), activation=act)
        out = {"y": y, "state_T": state}
        if op == "conv_train":
            grads = efla.causal_conv_bwd(*args, st["state0"], st["dy"], st["dstate_T"], activation=act)
            out |= {k: grads[k] for k in ("dx", "dstate0", "dw", "dbias") if grads[k] is not None}
        return out
    args = [st[k] for k in ("x", "dt", "A_log", "Bm", "Cm", "D", "dt_bias", "z")]
    if op == "scan_step":
        return {"y": efla.ssm_step(*args, st["state"]), "S": st["state"]}
    if op == "scan_train":
        y, S, ws = efla.ssm_scan_train(*args, st["state0"])
        grads = efla.ssm_scan_bwd(*args, st["state0"], st["dy"], st["dS_T"], workspace=ws, saved=True)
        names = ("dz", "dx", "ddt", "dB", "dC", "dA_log", "dD", "ddt_bias", "dS0")
        return {"y": y, "S_T": S, **{k: grads[k] for k in names if grads[k] is not None}}
    y, S = efla.ssm_scan(*args, st["state0"], st.get("cu_seqlens"))
    return {"y": y, "S_T": S}


def run(state):
    return dict(sorted((_own(state) if own else _plain(state)).items()))


# ------------------------------------------------------------------------------------ what it cannot do without
def work(case):
    op, es = case["op"], 2 if case["dtype"] == "bf16" else 4
    if op == "norm":
        n = case["rows"] * case["L"] * case["C"]
        return {"bytes": n * es * (4 if case["grad"] else 2) + case["C"] * (16 if case["grad"] else 8),
                "flops": n * (30 if case["grad"] else 12)}
    D = case["D"]
    if op.endswith("step"):
        tok, rows = case["B"], case["B"]
    elif op.endswith("packed"):
        tok, rows = sum(_lens(case)), case["n"]
    else:
        tok, rows = case["B"] * case["T"], case["B"]
    train = op.endswith("train")
    states = 2 if op.endswith("step") or case.get("S0") else 1
    if op.startswith("conv"):
        W = case["W"]
        n = tok * D
        state = rows * (W - 1) * D * es
        par = D * (W + int(case["bias"])) * 4
        return {"bytes": n * es * (4 if train else 2) + state * (states + 2 * train) + par * (1 + train),
                "flops": n * (2 * W + 5 + (4 * W + 10 if train else 0))}
    N, G, z = case["N"], case["G"], int(case["z"])
    io = tok * (D * (3 + z) + 2 * G * N) * es + D * (N + 2) * 4  # x, dt, z, y, B, C and the parameters
    if train:  # dy, dx, ddt, dz, dB, dC and the parameters' gradients
        io += tok * (D * (3 + z) + 2 * G * N) * es + D * (N + 2) * 4
    state = rows * D * N * 4
    return {"bytes": io + state * (states + 2 * train), "flops": tok * D * (N * (7 + (17 if train else 0)) + 25)}


# ------------------------------------------------------------------------------------ 64 bits, by the definition
def _exact_conv(case, x, w, bias, before, dy=None, dend=None):
    """[B, T, D] behind `before` [B, W - 1, D] through torch's own convolution in 64 bits."""
    D, W = w.shape
    full = torch.cat([before, x], 1)
    s = torch.nn.functional.conv1d(full.transpose(1, 2), w.unsqueeze(1), bias, groups=D).transpose(1, 2)
    y = torch.nn.functional.silu(s) if case["act"] else s
    return y, full[:, full.shape[1] - (W - 1):]


def _exact_gates(d, case):
    rep = case["D"] // case["G"]
    delta = torch.nn.functional.softplus(d["dt"] + d["dt_bias"], threshold=1e9)
    return delta, d["A_log"].exp().neg(), d["Bm"].repeat_interleave(rep, -2), d["Cm"].repeat_interleave(rep, -2)


def _exact_scan(d, case, sl, h, keep=False):
    """The recurrence over [B, T, ...] tokens `sl` of every row, one after the other."""
    delta, A, Bm, Cm = _exact_gates({k: v[:, sl] if k in ("x", "dt", "Bm", "Cm") else v for k, v in d.items()}, case)
    x = d["x"][:, sl]
    ys, hs = [], [h]
    for t in range(x.shape[1]):
        h = h * torch.exp(A * delta[:, t].unsqueeze(-1)) + Bm[:, t] * (delta[:, t] * x[:, t]).unsqueeze(-1)
        ys.append(torch.einsum("bdn,bdn->bd", h, Cm[:, t]))
        if keep:
            hs.append(h)
    y = torch.stack(ys, 1) + d["D"] * x
    if "z" in d:
        y = y * torch.nn.functional.silu(d["z"][:, sl])
    return y, h, ys, hs


def _exact_scan_train(d, case, h0):
    """Reverse mode of the recurrence, written for one token at a time."""
    D, N, G = case["D"], case["N"], case["G"]
    y, h_T, ys, hs = _exact_scan(d, case, slice(None), h0, keep=True)
    delta, A, Bm, Cm = _exact_gates(d, case)
    x, g = d["x"], d["dy"]
    out = {"y": y, "S_T": h_T}
    if "z" in d:
        s = torch.sigmoid(d["z"])
        out["dz"] = g * (torch.stack(ys, 1) + d["D"] * x) * (s + d["z"] * s * (1 - s))
        g = g * d["z"] * s
    dx, ddelta, dBs, dCs = [], [], [], []
    dA, lam = torch.zeros_like(h0), d["dS_T"]
    for t in range(x.shape[1] - 1, -1, -1):
        lam = lam + g[:, t].unsqueeze(-1) * Cm[:, t]
        dCs.append(hs[t + 1] * g[:, t].unsqueeze(-1))
        dBs.append(lam * (delta[:, t] * x[:, t]).unsqueeze(-1))
        into = torch.einsum("bdn,bdn->bd", lam, Bm[:, t])
        decay = torch.exp(A * delta[:, t].unsqueeze(-1))
        via = lam * decay * hs[t]
        dx.append(into * delta[:, t])
        ddelta.append(into * x[:, t] + torch.einsum("bdn,dn->bd", via, A))
        dA = dA + via * delta[:, t].unsqueeze(-1)
        lam = lam * decay
    stack = lambda m: torch.stack(m[::-1], 1)  # noqa: E731
    out["dx"] = stack(dx) + d["D"] * g
    out["ddt"] = stack(ddelta) * torch.sigmoid(d["dt"] + d["dt_bias"])
    out["dB"], out["dC"] = (stack(m).unflatten(2, (G, D // G)).sum(3) for m in (dBs, dCs))
    out["dA_log"], out["dD"] = dA.sum(0) * A, (g * x).sum((0, 1))
    out["ddt_bias"], out["dS0"] = out["ddt"].sum((0, 1)), lam
    return out


def exact(case, seed):
    return dict(sorted(_exact(case, seed).items()))


def _exact(case, seed):
    st = prepare(case, seed)
    op, d = st["op"], {k: v.double() for k, v in st.items() if torch.is_tensor(v) and v.is_floating_point()}
    if op == "norm":
        leaves = [d[k].requires_grad_() for k in ("x", "w", "b")]
        x, w, b = leaves
        rows, L, C = x.shape
        with torch.enable_grad():
            xg = x.reshape(rows, L, case["groups"], C // case["groups"])
            var, mean = torch.var_mean(xg, (1, 3), correction=0, keepdim=True)
            s = ((xg - mean) / torch.sqrt(var + EPS)).reshape(rows, L, C) * w + b
            y = torch.nn.functional.silu(s) if case["act"] else s
            out = {"y": y.detach()}
            if case["grad"]:
                out |= dict(zip(("dx", "dw", "db"), torch.autograd.grad(y, leaves, d["dy"])))
        return out
    if op.startswith("conv"):
        D, W = d["w"].shape
        if op == "conv_step":
            y, state = _exact_conv(case, d["x"].unsqueeze(1), d["w"], d.get("bias"), d["state"])
            return {"y": y.squeeze(1), "state": state}
        rows = len(st["lens"]) if op == "conv_packed" else case["B"]
        before = d["state0"] if "state0" in d else torch.zeros(rows, W - 1, D, dtype=torch.float64, device="cuda")
        if op == "conv_packed":
            cuts = [0, *np.cumsum(st["lens"]).tolist()]
            parts = [_exact_conv(case, d["x"][:, a:b], d["w"], d.get("bias"), before[i:i + 1])
                     for i, (a, b) in enumerate(zip(cuts, cuts[1:]))]
            return {"y": torch.cat([p[0] for p in parts], 1), "state_T": torch.cat([p[1] for p in parts])}
        if op == "conv":
            y, state = _exact_conv(case, d["x"], d["w"], d.get("bias"), before)
            return {"y": y, "state_T": state}
        names = [k for k in ("x", "w", "bias") if k in d]
        leaves = [d[k].requires_grad_() for k in names] + [before.requires_grad_()]
        with torch.enable_grad():
            y, state = _exact_conv(case, d["x"], d["w"], d.get("bias"), before)
            grads = torch.autograd.grad([y, state], leaves, [d["dy"], d["dstate_T"]])
        return {"y": y.detach(), "state_T": state.detach(),
                **{"d" + k: g for k, g in zip((*names, "state0"), grads)}}
    if op == "scan_step":
        d |= {k: d[k].unsqueeze(1) for k in ("x", "dt", "Bm", "Cm", "z") if k in d}
        y, h, _, _ = _exact_scan(d, case, slice(None), d["state"])
        return {"y": y.squeeze(1), "S": h}
    rows = len(st["lens"]) if op == "scan_packed" else case["B"]
    h = d["state0"] if "state0" in d else torch.zeros(rows, case["D"], case["N"], dtype=torch.float64, device="cuda")
    if op == "scan_train":
        return _exact_scan_train(d, case, h)
    if op == "scan_packed":
        cuts = [0, *np.cumsum(st["lens"]).tolist()]
        parts = [_exact_scan(d, case, slice(a, b), h[i:i + 1])[:2] for i, (a, b) in enumerate(zip(cuts, cuts[1:]))]
        return {"y": torch.cat([p[0] for p in parts], 1), "S_T": torch.cat([p[1] for p in parts])}
    y, h = _exact_scan(d, case, slice(None), h)[:2]
    return {"y": y, "S_T": h}
