"""Gated delta rule and the norms around it on the GPU against the 64-bit oracle (oracle/gated.py).

Tolerances, relative to the 2-norm and to the largest value of an output:
  fp32 on CUDA cores   an output is a chain of sums of d_k, 64, d_k and 64 products (K S, T'' R, Q S,
                       P U), each rounding by at most 2^-24 a term; a gradient is twice as long.  What
                       comes from earlier chunks is contracted by the decay and by I - alpha k k^T.
  tensor cores         operands that are not exact bf16 are two rounded bf16 parts: 2^-18 off at most,
                       and the product of two low parts, left out, is 2^-18 at most; 8 such in the
                       chain of an output, 16 in a gradient's.
  bf16 outputs         half a step more: 2^-8 of the value.
"""
import math

import pytest
import torch

import exact_delta_rule_gb300 as efla
from oracle import gated

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def tol(dtype, dk, dv, grad=False):
    links = 2 if grad else 1
    t = links * 2 * (dk + 64) * 2.0 ** -24
    if dtype == BF16:
        t += links * 8 * 2.0 ** -18
    return t


def close(got, ref, t, what=""):
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    step = 2.0 ** -8 if got.dtype == BF16 else 0.0
    got, ref = got.double(), ref.double().to(got.device)
    assert bool(torch.isfinite(got).all()), f"{what}: non-finite values"
    if not ref.numel():
        return
    d = (got - ref).abs()
    worst = float((d - step * ref.abs() - t * ref.abs().max()).max())
    assert worst <= 0, f"{what}: {float(d.max()):.3e} off, largest value {float(ref.abs().max()):.3e}, tolerance {t:.1e}"
    norm = float(ref.norm())
    assert float(d.norm()) <= (t + step) * norm, f"{what}: rel {float(d.norm()) / max(norm, 1e-300):.3e}, tolerance {t + step:.1e}"


def make(B=2, T=70, Hk=2, H=4, dk=64, dv=64, dtype=F32, S0=True, N=None, seed=0, norm=1.0, rate=None):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    rate = torch.exp(r(H) - 1) if rate is None else rate
    return {"q": (unit(r(B, T, Hk, dk))).to(dtype), "k": (norm * unit(r(B, T, Hk, dk))).to(dtype), "v": r(B, T, H, dv).to(dtype),
            "g": -rate * torch.nn.functional.softplus(r(B, T, H)), "beta": torch.sigmoid(r(B, T, H)),
            "S0": 0.3 * r(B if N is None else N, H, dk, dv) if S0 else None}


def check_fwd(x, update="euler", **kw):
    o, S = efla.gated_fwd_chunked(**x, update=update, **kw)
    ref_o, ref_S = gated.fwd(**x, update=update)
    t = tol(x["q"].dtype, x["q"].shape[-1], x["v"].shape[-1])
    close(o, ref_o, t, "o")
    close(S, ref_S, t, "S_T")
    assert efla.device_status() == 0
    return o, S


SHAPES = [(F32, 32, 32), (F32, 64, 128), (F32, 128, 128), (BF16, 64, 64), (BF16, 128, 64), (BF16, 32, 128), (BF16, 128, 128)]


@pytest.mark.parametrize("T", [0, 1, 2, 15, 63, 64, 65, 127, 128, 130, 321])
@pytest.mark.parametrize("dtype, dk, dv", SHAPES)
def test_forward_lengths(dtype, dk, dv, T):
    check_fwd(make(T=T, dk=dk, dv=dv, dtype=dtype, seed=T))


@pytest.mark.parametrize("Hk, H", [(1, 1), (1, 5), (3, 3), (2, 6)])
@pytest.mark.parametrize("dtype, dk, dv", [(F32, 32, 64), (BF16, 128, 128)])
@pytest.mark.parametrize("update", ["euler", "exact"])
def test_forward_heads_and_rules(dtype, dk, dv, Hk, H, update):
    check_fwd(make(B=3, T=200, Hk=Hk, H=H, dk=dk, dv=dv, dtype=dtype, S0=False, norm=1.3 if update == "exact" else 1.0), update)


@pytest.mark.parametrize("dtype, d", [(F32, 64), (BF16, 128)])
def test_forward_options(dtype, d):
    x = make(T=150, dk=d, dv=d, dtype=dtype)
    o, S = check_fwd(x)
    for od in (BF16, F32):
        o2, _ = efla.gated_fwd_chunked(**x, o_dtype=od)
        close(o2, gated.fwd(**x)[0], tol(dtype, d, d), f"o as {od}")
    o2, none = efla.gated_fwd_chunked(**x, return_state=False)
    assert none is None and torch.equal(o, o2)
    inplace = {**x, "S0": x["S0"].clone()}  # S0 and S_T the same memory
    o2, S2 = efla.gated_fwd_chunked(**inplace, S_T=inplace["S0"])
    assert torch.equal(o2, o) and torch.equal(S2, S) and S2.data_ptr() == inplace["S0"].data_ptr()
    o3, S3, _ = efla.gated_fwd_chunked_train(**x)  # the training forward gives the same bits
    assert torch.equal(o3, o) and torch.equal(S3, S)


@pytest.mark.parametrize("dtype, d", [(F32, 64), (BF16, 128)])
def test_forward_is_causal_and_splits(dtype, d):
    """A prefix does not see what follows it, and a state handed over continues the sequence."""
    x = make(T=200, dk=d, dv=d, dtype=dtype)
    o, S = efla.gated_fwd_chunked(**x)
    for cut in (1, 64, 101):
        head = {n: t if n == "S0" else t[:, :cut].contiguous() for n, t in x.items()}
        o1, S1 = efla.gated_fwd_chunked(**head)
        tail = {n: S1 if n == "S0" else t[:, cut:].contiguous() for n, t in x.items()}
        o2, S2 = efla.gated_fwd_chunked(**tail)
        t = 2 * tol(dtype, d, d)
        close(torch.cat([o1, o2], 1).float(), o.double(), t + (2 ** -7 if dtype == BF16 else 0), "o")
        close(S2, S.double(), t, "S_T")


@pytest.mark.parametrize("dtype, dk, dv", [(F32, 32, 64), (BF16, 128, 128)])
def test_forward_packed(dtype, dk, dv):
    lens = [5, 0, 64, 1, 130, 0, 63, 200, 65]
    x = make(B=1, T=sum(lens), N=len(lens), dk=dk, dv=dv, dtype=dtype)
    cu = torch.tensor([0] + lens, dtype=torch.int32).cumsum(0).to(torch.int32).cuda()
    o, S = efla.gated_fwd_chunked(**x, cu_seqlens=cu)
    t = tol(dtype, dk, dv)
    for i, n in enumerate(lens):
        a = int(cu[i])
        part = {m: y[i:i + 1] if m == "S0" else y[:, a:a + n] for m, y in x.items()}
        ro, rS = gated.fwd(**part)
        close(o[:, a:a + n], ro, t, f"o of sequence {i}")
        close(S[i:i + 1], rS, t, f"S_T of sequence {i}")
    assert efla.device_status() == 0


@pytest.mark.parametrize("dtype, d", [(F32, 32), (BF16, 64), (BF16, 128)])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_forward_packed_keeps_bad_values_in_their_sequence(dtype, d, bad):
    lens = [70, 40, 64, 5]
    x = make(B=1, T=sum(lens), N=4, dk=d, dv=d, dtype=dtype)
    cu = torch.tensor([0, 70, 110, 174, 179], dtype=torch.int32, device="cuda")
    want_o, want_S = efla.gated_fwd_chunked(**x, cu_seqlens=cu)
    for n in ("q", "k", "v", "g", "beta"):
        x[n][:, 70:110] = -bad if n == "g" else bad
    x["S0"][1] = bad
    o, S = efla.gated_fwd_chunked(**x, cu_seqlens=cu)
    for a, b, i in ((0, 70, 0), (110, 174, 2), (174, 179, 3)):
        assert torch.equal(o[:, a:b], want_o[:, a:b]) and torch.equal(S[i], want_S[i]), i
    assert efla.device_status() == 0


@pytest.mark.parametrize("dtype, d", [(F32, 64), (BF16, 32), (BF16, 128)])
def test_rows_keep_bad_values_to_themselves(dtype, d):
    """A batch row of NaN leaves the other rows' outputs and gradients as they were, in every call."""
    x = make(B=3, T=70, dk=d, dv=d, dtype=dtype)
    dO, dS = torch.ones_like(x["v"]), torch.ones_like(x["S0"])
    S1, S2 = x["S0"].clone(), x["S0"].clone()
    tok = lambda x, n: [x[m][:, :n].contiguous() for m in ("q", "k", "v", "g", "beta")]  # noqa: E731
    run = lambda x, dO, S1, S2: [*efla.gated_fwd_chunked(**x), *efla.gated_bwd_chunked(*x.values(), dO, dS).values(),  # noqa: E731
                                 efla.gated_decode_tokens(*tok(x, 19), S1), S1,
                                 efla.gated_decode_step(*[t[:, 0].contiguous() for t in tok(x, 1)], S2), S2]
    want = run(x, dO, S1, S2)
    S1, S2 = x["S0"].clone(), x["S0"].clone()
    for t in (*x.values(), dO, S1, S2):
        t[1] = math.nan
    for got, ref in zip(run(x, dO, S1, S2), want):
        assert torch.equal(got[[0, 2]], ref[[0, 2]])


def test_positive_gates():
    x = make(B=1, T=150, dk=64, dv=64, dtype=BF16)
    x["g"].mul_(-0.01)
    check_fwd(x)
    check_bwd(x)


@pytest.mark.parametrize("dtype, d", [(F32, 32), (BF16, 128)])
def test_forward_packed_bad_bounds_are_flagged(dtype, d):
    """A sequence with bounds outside the tokens is not touched; the others are computed."""
    x = make(B=1, T=100, N=3, dk=d, dv=d, dtype=dtype)
    for bounds in ([0, 40, 200, 100], [0, 60, 30, 100], [-5, 10, 40, 100]):
        cu = torch.tensor(bounds, dtype=torch.int32, device="cuda")
        S_T = torch.full((3, 4, d, d), 7.0, device="cuda")
        o = torch.full((1, 100, 4, d), 7.0, device="cuda", dtype=dtype)
        efla.gated_fwd_chunked(**x, cu_seqlens=cu, o=o, S_T=S_T)
        assert efla.device_status() == 1
        for n in range(3):
            a, b = bounds[n], bounds[n + 1]
            if a < 0 or b < a or b > 100:
                assert bool((S_T[n] == 7).all())
        assert efla.device_status() == 0


@pytest.mark.parametrize("dtype, dk, dv", [(F32, 64, 64), (F32, 32, 128), (BF16, 128, 128), (BF16, 32, 64), (BF16, 128, 32)])
@pytest.mark.parametrize("what", ["none", "resets", "strong", "weak", "zero keys", "zero beta", "one beta", "same key"])
def test_forward_extremes(dtype, dk, dv, what):
    x = make(B=1, T=190, dk=dk, dv=dv, dtype=dtype, seed=3)
    g, beta, k = x["g"], x["beta"], x["k"]
    if what == "none":
        g.zero_()
    elif what == "resets":  # documents that begin inside the sequence, one at a chunk's first token, a run of them
        g[:, [0, 10, 64, 65, 66, 150]] = -math.inf
        g[:, 100] = -1e30
    elif what == "strong":
        g.mul_(0).sub_(20.0)
    elif what == "weak":
        g.mul_(1e-4)
    elif what == "zero keys":
        k[:, ::3] = 0
    elif what == "zero beta":
        beta[:, ::2] = 0
    elif what == "one beta":
        beta.fill_(1.0)
    else:
        k[:] = k[:, :1]
    check_fwd(x)
    check_fwd(x, "exact")


def test_forward_reset_equals_a_new_sequence():
    x = make(B=1, T=150, dk=128, dv=128, dtype=BF16, S0=False)
    x["g"][:, 70] = -math.inf
    o, S = efla.gated_fwd_chunked(**x)
    tail = {n: None if t is None else t[:, 70:].contiguous() for n, t in x.items()}
    o2, S2 = efla.gated_fwd_chunked(**tail)
    close(S, S2.double(), 2 * tol(BF16, 128, 128), "S_T")
    close(o[:, 70:].float(), o2.double(), 2 * tol(BF16, 128, 128) + 2 ** -7, "o")


@pytest.mark.parametrize("dtype, d", [(F32, 64), (BF16, 128)])
def test_calls_write_only_their_outputs(dtype, d):
    """Outputs inside larger buffers: nothing before or behind them changes, and a repeat gives the same bits."""
    x = make(B=2, T=90, dk=d, dv=d, dtype=dtype)
    n_o, n_s = 2 * 90 * 4 * d, 2 * 4 * d * d
    bo, bs = torch.full((n_o + 512,), 3.0, dtype=dtype, device="cuda"), torch.full((n_s + 512,), 3.0, device="cuda")
    o, S = efla.gated_fwd_chunked(**x, o=bo[256:256 + n_o].view(2, 90, 4, d), S_T=bs[256:256 + n_s].view(2, 4, d, d))
    for b, n in ((bo, n_o), (bs, n_s)):
        assert bool((b[:256] == 3).all()) and bool((b[256 + n:] == 3).all())
    o2, S2 = efla.gated_fwd_chunked(**x)
    assert torch.equal(o, o2) and torch.equal(S, S2)


# ------------------------------------------------------------------------------ backward
def check_bwd(x, update="euler", dS=True, saved=True, seed=5):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dO = torch.randn(x["v"].shape, generator=gen, device="cuda").to(x["q"].dtype)
    B, _, H, dv = x["v"].shape
    dk = x["q"].shape[-1]
    dS_T = torch.randn((B, H, dk, dv), generator=gen, device="cuda") if dS else None
    ws = efla.gated_fwd_chunked_train(**x, update=update)[2] if saved else None
    got = efla.gated_bwd_chunked(*x.values(), dO, dS_T, workspace=ws, saved=saved, update=update)
    ref = gated.bwd(*x.values(), dO, dS_T, update)
    assert efla.device_status() == 0
    for n, r in ref.items():
        close(got[n], r, tol(x["q"].dtype, dk, dv, True), n)
    return got


@pytest.mark.parametrize("T", [0, 1, 2, 63, 64, 65, 129, 200])
@pytest.mark.parametrize("dtype, dk, dv", SHAPES)
def test_backward_lengths(dtype, dk, dv, T):
    check_bwd(make(T=T, dk=dk, dv=dv, dtype=dtype, seed=T))


@pytest.mark.parametrize("Hk, H", [(1, 1), (1, 5), (3, 3), (2, 6)])
@pytest.mark.parametrize("dtype, dk, dv", [(F32, 32, 64), (BF16, 128, 128)])
@pytest.mark.parametrize("update", ["euler", "exact"])
def test_backward_heads_and_rules(dtype, dk, dv, Hk, H, update):
    x = make(B=2, T=140, Hk=Hk, H=H, dk=dk, dv=dv, dtype=dtype, S0=False, norm=1.3 if update == "exact" else 1.0)
    check_bwd(x, update, dS=False, saved=False)


@pytest.mark.parametrize("dtype, dk, dv", [(F32, 64, 64), (BF16, 128, 128), (BF16, 64, 128), (BF16, 32, 32)])
@pytest.mark.parametrize("what", ["none", "strong", "weak", "zero keys", "zero beta", "one beta", "resets"])
def test_backward_extremes(dtype, dk, dv, what):
    x = make(B=1, T=190, dk=dk, dv=dv, dtype=dtype, seed=3)
    if what == "none":
        x["g"].zero_()
    elif what == "strong":
        x["g"].mul_(0).sub_(20.0)
    elif what == "weak":
        x["g"].mul_(1e-4)
    elif what == "zero keys":
        x["k"][:, ::3] = 0
    elif what == "zero beta":
        x["beta"][:, ::2] = 0
    elif what == "one beta":
        x["beta"].fill_(1.0)
    else:
        x["g"][:, [0, 10, 64, 150]] = -1000.0
    check_bwd(x)
    if what in ("none", "zero keys"):
        check_bwd(x, "exact")


@pytest.mark.parametrize("dtype, d", [(F32, 64), (BF16, 128)])
def test_backward_repeats_bit_for_bit(dtype, d):
    x = make(T=150, dk=d, dv=d, dtype=dtype)
    a, b, c = check_bwd(x), check_bwd(x), check_bwd(x, saved=False)
    for n in a:
        assert torch.equal(a[n], b[n]) and torch.equal(a[n], c[n]), n


def test_backward_without_dS0():
    x = make(T=70)
    dO = torch.ones_like(x["v"])
    got = efla.gated_bwd_chunked(*x.values(), dO, need_dS0=False)
    want = efla.gated_bwd_chunked(*x.values(), dO)
    assert got["dS0"] is None and all(torch.equal(got[n], want[n]) for n in got if n != "dS0")


# ------------------------------------------------------------------------------ decode
@pytest.mark.parametrize("B", [1, 3, 40])
@pytest.mark.parametrize("m", [0, 1, 2, 15, 16, 17, 40])
@pytest.mark.parametrize("dtype, dk, dv", [(F32, 32, 64), (F32, 128, 128), (BF16, 64, 32), (BF16, 128, 128)])
def test_decode_tokens(dtype, dk, dv, m, B):
    x = make(B=B, T=m, dk=dk, dv=dv, dtype=dtype, seed=m)
    S = x.pop("S0")
    ref_o, ref_S = gated.fwd(**x, S0=S)
    S1 = S.clone()
    o = efla.gated_decode_tokens(**x, S=S1)
    close(o, ref_o, tol(dtype, dk, dv), "o")
    close(S1, ref_S, tol(dtype, dk, dv), "S")
    if 0 < m <= 17:  # the same by single steps
        S2, outs = S.clone(), []
        for t in range(m):
            outs.append(efla.gated_decode_step(**{n: y[:, t].contiguous() for n, y in x.items()}, S=S2))
        close(torch.stack(outs, 1), ref_o, tol(dtype, dk, dv), "o by steps")
        close(S2, ref_S, tol(dtype, dk, dv), "S by steps")
    assert efla.device_status() == 0


@pytest.mark.parametrize("B, Hk, H", [(1, 1, 1), (400, 1, 1), (160, 1, 2), (2, 3, 9)])
@pytest.mark.parametrize("dk", [32, 64, 128])
@pytest.mark.parametrize("dv", [32, 64, 128])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_decode_step_shapes(dtype, dk, dv, B, Hk, H):
    x = make(B=B, T=1, Hk=Hk, H=H, dk=dk, dv=dv, dtype=dtype)
    S = x.pop("S0")
    for update in ("euler", "exact"):
        ref_o, ref_S = gated.fwd(**x, S0=S, update=update)
        S1 = S.clone()
        o = efla.gated_decode_step(**{n: y[:, 0].contiguous() for n, y in x.items()}, S=S1, update=update, o_dtype=F32)
        close(o, ref_o[:, 0], tol(F32, dk, dv), "o")
        close(S1, ref_S, tol(F32, dk, dv), "S")


@pytest.mark.parametrize("dtype, d", [(F32, 64), (BF16, 128)])
def test_decode_resets(dtype, d):
    x = make(B=2, T=20, dk=d, dv=d, dtype=dtype)
    x["g"][:, [0, 7]] = -math.inf
    S = x.pop("S0")
    ref_o, ref_S = gated.fwd(**x, S0=S)
    o = efla.gated_decode_tokens(**x, S=S)
    close(o, ref_o, tol(dtype, d, d), "o")
    close(S, ref_S, tol(dtype, d, d), "S")


# ------------------------------------------------------------------------------ norms
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("lead, Hk, H, dk", [((1, 1), 1, 1, 32), ((2, 3), 2, 4, 64), ((1, 517), 3, 7, 128), ((4,), 16, 33, 128),
                                             ((0,), 2, 2, 64), ((3, 300), 1, 70, 32)])
def test_prep(dtype, lead, Hk, H, dk):
    gen = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    q, k = r(*lead, Hk, dk).to(dtype), (3 * r(*lead, Hk, dk)).to(dtype)
    a, b = (4 * r(*lead, H)).to(dtype), (4 * r(*lead, H)).to(dtype)
    if q.numel():
        q[..., 0, :] = 0  # a zero row: 0 / sqrt(eps)
        a.view(-1)[0], b.view(-1)[0] = 60.0, -60.0  # saturated gates
    A, d = r(H), r(H)
    # sums of dk squares, then a handful of roundings; exp, log and the square root are within 2 steps
    t = (dk + 16) * 2.0 ** -24
    got, ref = efla.gated_prep(q, k, a, b, A, d, scale=0.25), gated.prep(q, k, a, b, A, d, 0.25)
    for n in ref:
        close(got[n], ref[n], t, n)
    dys = [r(*x.shape).to(x.dtype) for x in got.values()]
    got, ref = efla.gated_prep_bwd(q, k, a, b, A, d, *dys, scale=0.25), gated.prep_bwd(q, k, a, b, A, d, *dys, 0.25)
    tokens = math.prod(lead)
    for n in ref:  # a token's sum is rounded once a term: 2^-24 of the terms' sizes, whose sum may be small
        close(got[n], ref[n], (2 * t + max(tokens, 1) ** 0.5 * 2.0 ** -22) if n in ("dA_log", "ddt_bias") else 2 * t, n)
    again = efla.gated_prep_bwd(q, k, a, b, A, d, *dys, scale=0.25)
    assert all(torch.equal(got[n], again[n]) for n in got)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", [(1, 32), (3, 64), (7, 5, 128), (2, 1111, 3, 64), (0, 128), (130, 32), (40000, 128)])
def test_norm_gate(dtype, shape):
    gen = torch.Generator(device="cuda").manual_seed(2)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    o, z, w = (2 * r(*shape)).to(dtype), (3 * r(*shape)).to(dtype), r(shape[-1])
    if o.numel():
        o.view(-1, shape[-1])[0] = 0
        z.view(-1)[0], z.view(-1)[-1] = 80.0, -80.0
    t = (shape[-1] + 16) * 2.0 ** -24
    y = efla.norm_gate(o, z, w)
    close(y, gated.norm_gate(o, z, w), t, "y")
    for alias in (o, z):  # in place
        c = alias.clone()
        args = (c, z, w) if alias is o else (o, c, w)
        assert torch.equal(efla.norm_gate(*args, y=c), y)
    dy = r(*shape).to(dtype)
    got, ref = efla.norm_gate_bwd(o, z, w, dy), gated.norm_gate_bwd(o, z, w, dy)
    rows = max(1, math.prod(shape[:-1]))
    if rows > 0 and o.numel():  # a zero row has a gradient of size 1 / sqrt(eps): compared by itself
        close(got["do"].view(-1, shape[-1])[:1], ref["do"].view(-1, shape[-1])[:1], 2 * t, "do of the zero row")
        close(got["do"].view(-1, shape[-1])[1:], ref["do"].view(-1, shape[-1])[1:], 2 * t, "do")
    close(got["dz"], ref["dz"], 2 * t, "dz")
    close(got["dw"], ref["dw"], 2 * t + rows ** 0.5 * 2.0 ** -22, "dw")
    again = efla.norm_gate_bwd(o, z, w, dy)
    assert all(torch.equal(got[n], again[n]) for n in got)


# ------------------------------------------------------------------------------ together
@pytest.mark.parametrize("dtype, dk, dv", [(F32, 64, 32), (BF16, 128, 128)])
def test_a_mixer_trains_and_decodes(dtype, dk, dv):
    """Norms and gates, the rule, the gated output norm: gradients of the run against the oracle's
    (from the same rounded values between the operators), and the same tokens one by one."""
    B, T, Hk, H = 2, 100, 2, 4
    gen = torch.Generator(device="cuda").manual_seed(4)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    q, k, v, z = (r(B, T, n, d).to(dtype) for n, d in ((Hk, dk), (Hk, dk), (H, dv), (H, dv)))
    a, b, A, bias, w = r(B, T, H).to(dtype), r(B, T, H).to(dtype), r(H), r(H) - 2, 1 + 0.1 * r(dv)
    p = efla.gated_prep(q, k, a, b, A, bias, scale=dk ** -0.5)
    o, S, ws = efla.gated_fwd_chunked_train(p["q"], p["k"], v, p["g"], p["beta"])
    y = efla.norm_gate(o, z, w)
    dy = r(B, T, H, dv).to(dtype)
    dn = efla.norm_gate_bwd(o, z, w, dy)
    dm = efla.gated_bwd_chunked(p["q"], p["k"], v, p["g"], p["beta"], None, dn["do"], workspace=ws, saved=True)
    dp = efla.gated_prep_bwd(q, k, a, b, A, bias, dm["dq"], dm["dk"], dm["dg"], dm["dbeta"], scale=dk ** -0.5)
    t = tol(dtype, dk, dv, True) + (dk + 16) * 2.0 ** -23
    ro, rS = gated.fwd(p["q"], p["k"], v, p["g"], p["beta"])
    close(S, rS, t, "S")
    close(y, gated.norm_gate(o, z, w), t, "y")
    rn = gated.norm_gate_bwd(o, z, w, dy)
    rm = gated.bwd(p["q"], p["k"], v, p["g"], p["beta"], None, dn["do"])
    rp = gated.prep_bwd(q, k, a, b, A, bias, dm["dq"], dm["dk"], dm["dg"], dm["dbeta"], dk ** -0.5)
    for got, ref in ((dn, rn), (dm, rm), (dp, rp)):
        for n in ref:
            close(got[n], ref[n], t + (T * B) ** 0.5 * 2.0 ** -22, n)
    S1 = torch.zeros_like(S)
    for i in range(T):
        x = efla.gated_prep(q[:, i].contiguous(), k[:, i].contiguous(), a[:, i].contiguous(), b[:, i].contiguous(), A, bias,
                            scale=dk ** -0.5)
        assert torch.equal(x["q"], p["q"][:, i]) and torch.equal(x["g"], p["g"][:, i])
        o1 = efla.gated_decode_step(x["q"], x["k"], v[:, i].contiguous(), x["g"], x["beta"], S1)
        close(o1, ro[:, i], t, f"o of token {i}")
    close(S1, rS, t, "S by steps")


def test_captured_calls_replay():
    """Every call captured into one graph and replayed on new inputs gives the eager results."""
    def run(x, S, dO):
        p = efla.gated_prep(x["q"], x["k"], x["a"], x["b"], x["A"], x["bias"], scale=0.5)
        o, S_T, ws = efla.gated_fwd_chunked_train(p["q"], p["k"], x["v"], p["g"], p["beta"])
        d = efla.gated_bwd_chunked(p["q"], p["k"], x["v"], p["g"], p["beta"], None, dO, workspace=ws, saved=True)
        e = efla.gated_prep_bwd(x["q"], x["k"], x["a"], x["b"], x["A"], x["bias"], d["dq"], d["dk"], d["dg"], d["dbeta"])
        y = efla.norm_gate(o, dO, x["w"])
        n = efla.norm_gate_bwd(o, dO, x["w"], y)
        t = efla.gated_decode_tokens(p["q"], p["k"], x["v"], p["g"], p["beta"], S)
        return [o, S_T, y, t, *d.values(), *e.values(), *n.values()]

    def fresh(seed):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        r = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
        x = {"q": r(2, 80, 2, 128).bfloat16(), "k": r(2, 80, 2, 128).bfloat16(), "v": r(2, 80, 4, 128).bfloat16(),
             "a": r(2, 80, 4).bfloat16(), "b": r(2, 80, 4).bfloat16(), "A": r(4), "bias": r(4), "w": r(128)}
        return x, r(2, 4, 128, 128), r(2, 80, 4, 128).bfloat16()

    x, S, dO = fresh(0)
    S_graph = S.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(x, S.clone(), dO)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run(x, S_graph, dO)
    for seed in (1, 2):
        x2, S2, dO2 = fresh(seed)
        for n in x:
            x[n].copy_(x2[n])
        S_graph.copy_(S2)
        dO.copy_(dO2)
        graph.replay()
        for got, want in zip(out + [S_graph], run(x2, S2, dO2) + [S2]):
            assert torch.equal(got, want)


def test_streams():
    """A call on another stream than the current one, its outputs and workspace allocated here."""
    x = make(T=300, dk=128, dv=128, dtype=BF16)
    dO = torch.ones_like(x["v"])
    want_o, want_S = efla.gated_fwd_chunked(**x)
    want = efla.gated_bwd_chunked(*x.values(), dO)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    o, S = efla.gated_fwd_chunked(**x, stream=side)
    got = efla.gated_bwd_chunked(*x.values(), dO, stream=side)
    junk = [torch.full((1 << 20,), 9.0, device="cuda") for _ in range(8)]  # reuses whatever was freed too early
    side.synchronize()
    assert torch.equal(o, want_o) and torch.equal(S, want_S)
    assert all(torch.equal(got[n], want[n]) for n in got), len(junk)


def test_stream_outputs_wait_for_their_memory():
    """An output on another stream does not land in memory that the current stream is still writing."""
    x = make(T=300, dk=128, dv=128, dtype=BF16)
    want_o, want_S = efla.gated_fwd_chunked(**x)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    side = torch.cuda.Stream()
    late = [torch.empty_like(want_o), torch.empty_like(want_S)]
    torch.cuda._sleep(100_000_000)  # the writes below happen long after the call on the other stream
    for t in late:
        t.fill_(7.0)
    del late, t
    o, S = efla.gated_fwd_chunked(**x, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(o, want_o) and torch.equal(S, want_S)


def test_two_graphs_and_an_eager_call_share_a_workspace():
    """Replayed in turn on one stream, each graph's forward fills the workspace before its backward reads it."""
    xs = [make(T=n, dk=64, dv=128, dtype=BF16, seed=n) for n in (130, 190)]
    ws = torch.empty(max(efla.gated_bwd_workspace(2, n, 2, 4, 64, 128, BF16) for n in (130, 190)), dtype=torch.uint8,
                     device="cuda")
    dO = [torch.ones_like(x["v"]) for x in xs]
    step = lambda i: efla.gated_bwd_chunked(*xs[i].values(), dO[i], workspace=ws)  # noqa: E731
    want = [{n: t.clone() for n, t in step(i).items()} for i in (0, 1)]
    torch.cuda.synchronize()
    graphs, got = [], []
    for i in (0, 1):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i]):
            got.append(step(i))
    for i in (0, 1, 1, 0):
        graphs[i].replay()
        eager = step(1 - i)
        torch.cuda.synchronize()
        for n in want[i]:
            assert torch.equal(got[i][n], want[i][n]) and torch.equal(eager[n], want[1 - i][n]), n


@pytest.mark.parametrize("stall", [1, 2, 4])
@pytest.mark.parametrize("T", [64, 200])
def test_expired_waits_are_reported(stall, T):
    """A wait that runs out in the forward, the state pass or the gradient pass: the kernel records it and
    leaves, and the next call is right."""
    x = make(B=1, T=T, dk=128, dv=64, dtype=BF16)
    dO = torch.ones_like(x["v"])
    assert efla.device_status() == 0
    efla.set_wait_limit_ns(50_000_000)
    efla.set_debug_stall(stall)
    try:
        efla.gated_bwd_chunked(*x.values(), dO)
        torch.cuda.synchronize()
    finally:
        efla.set_debug_stall(False)
        efla.set_wait_limit_ns(0)
    assert efla.device_status() == 4
    assert efla.device_status() == 0
    check_fwd(x)
    check_bwd(x)


@pytest.mark.parametrize("dk, dv", [(32, 128), (64, 32), (128, 64)])
def test_small_heads_touch_only_their_memory(dk, dv):
    """Head sizes that the tensor-core tiles exceed, every output between sentinels; partial chunks, packed too."""
    T, H, N = 70, 4, 2
    x = make(B=1, T=T, dk=dk, dv=dv, dtype=BF16, N=N)
    cu = torch.tensor([0, 33, 66], dtype=torch.int32, device="cuda")  # (four tokens behind the last sequence)
    big = torch.full((64 + T * H * dv + 64,), 7.0, device="cuda", dtype=BF16)
    bigS = torch.full((64 + N * H * dk * dv + 64,), 7.0, device="cuda")
    o, S = big[64:-64].view(1, T, H, dv), bigS[64:-64].view(N, H, dk, dv)
    efla.gated_fwd_chunked(**x, cu_seqlens=cu, o=o, S_T=S)
    ref = [gated.fwd(**{m: y[i:i + 1] if m == "S0" else y[:, 33 * i:33 * i + 33] for m, y in x.items()}) for i in (0, 1)]
    t = tol(BF16, dk, dv)
    close(o[:, :66], torch.cat([r[0] for r in ref], 1), t, "o")
    close(S, torch.cat([r[1] for r in ref]), t, "S_T")
    assert all(bool((e == 7).all()) for e in (big[:64], big[-64:], bigS[:64], bigS[-64:], o[:, 66:]))
    y = make(B=2, T=T, Hk=4, H=4, dk=dk, dv=dv, dtype=BF16)
    check_fwd(y)
    check_fwd(y, o_dtype=F32)
    check_bwd(y)


@pytest.mark.parametrize("dtype, d", [(F32, 64), (BF16, 128)])
def test_long_sequence(dtype, d):
    """4096 tokens, weak and strong decays side by side: errors do not pile up."""
    rate = torch.tensor([1e-3, 2.0], device="cuda")
    x = make(B=1, T=4096, Hk=1, H=2, dk=d, dv=d, dtype=dtype, rate=rate)
    check_fwd(x)
    check_bwd(x)


def test_many_heads():
    """More (sequence, head) units than one wave of CTAs."""
    x = make(B=40, T=66, Hk=4, H=8, dk=128, dv=128, dtype=BF16)
    check_fwd(x)
    check_bwd(x)


def test_offsets_past_32_bits():
    """States, values and rows of more than 2^31 elements: the last of them against the same call on them alone."""
    last = lambda *ts: [t[-1:].contiguous() for t in ts]  # noqa: E731
    gen = torch.Generator(device="cuda").manual_seed(0)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    B, H, d = 3300, 40, 128  # 2^31 + 15 M elements of S
    q, v, g, beta = r(B, H, d).bfloat16() / 12, r(B, H, d).bfloat16(), -r(B, H).abs(), torch.sigmoid(r(B, H))
    S = torch.zeros(B, H, d, d, device="cuda")
    S[-1] = r(H, d, d)
    assert S.numel() > 2 ** 31
    few = S[-33:].clone()  # (as many heads as take the same kernel variant)
    x = [t[-33:].contiguous() for t in (q, q, v, g, beta)]
    o, want = efla.gated_decode_step(q, q, v, g, beta, S), efla.gated_decode_step(*x, few)
    assert torch.equal(o[-33:], want) and torch.equal(S[-33:], few)
    o = efla.gated_decode_tokens(*(t[:, None].contiguous() for t in (q, q, v, g, beta)), S)
    want = efla.gated_decode_tokens(*(t[:, None].contiguous() for t in x), few)
    assert torch.equal(o[-33:], want) and torch.equal(S[-33:], few)
    del S, o
    rows = 2 ** 24 + 3
    z, w = r(4096, d).bfloat16().repeat(rows // 4096 + 1, 1)[:rows], r(d)
    assert z.numel() > 2 ** 31
    got, want = efla.norm_gate_bwd(z, z, w, z), efla.norm_gate_bwd(*last(z, z), w, *last(z))
    assert torch.equal(got["do"][-1:], want["do"]) and torch.equal(got["dz"][-1:], want["dz"])
    assert torch.equal(efla.norm_gate(z, z, w)[-1:], efla.norm_gate(*last(z, z), w))
    del got
    heads = z[:rows // 8 * 8].view(-1, 8, d)
    a = torch.zeros(heads.shape[0], 8, device="cuda", dtype=BF16)
    A = torch.zeros(8, device="cuda")
    p, want = efla.gated_prep(heads, heads, a, a, A, A), efla.gated_prep(*last(heads, heads, a, a), A, A)
    assert all(torch.equal(p[n][-1:], want[n]) for n in p)
    assert efla.device_status() == 0


# ------------------------------------------------------------------------------ decays inside a quarter of a chunk
def quarters(H, seed):
    """Gates of 64 tokens of H heads [1, 64, H]: by heads in turn, one strong gate in every 16 tokens among weak ones
    (2^64 to 2^100 of decay; 2^40 to 2^66), and a steady decay of 2^5.2 to 2^6.6 a token."""
    gen = torch.Generator().manual_seed(seed)
    u = lambda lo, hi, *s: lo + (hi - lo) * torch.rand(s, generator=gen, dtype=torch.float64)  # noqa: E731
    g = u(-0.3, 0.0, H, 4, 16)
    at = torch.randint(0, 16, (H, 4, 1), generator=gen)
    strong = torch.where(torch.arange(H)[:, None, None] % 3 == 0, u(-69.0, -45.0, H, 4, 1), u(-45.0, -28.0, H, 4, 1))
    g.scatter_(2, at, strong)
    g[2::3] = u(-4.6, -3.6, *g[2::3].shape)
    return g.reshape(H, 64).t()[None].float().contiguous().cuda()


def one_hot_tokens(H, d, seed):
    """k_t = e_t, v_t = e_t, q_t = 1, beta = 1: u_t = e_t without rounding, so that o_t[s] = Gamma_ts."""
    e = torch.eye(64, d, device="cuda", dtype=BF16)
    k = e[None, :, None]
    g = quarters(H, seed)
    G = g[0].double().cumsum(0).t()  # [H, 64]
    gamma = (G[:, :, None] - G[:, None, :]).tril().exp().tril()  # [H, t, s]
    x = {"q": torch.ones_like(k), "k": k, "v": e[None, :, None].expand(1, 64, H, d).contiguous(), "g": g,
         "beta": torch.ones_like(g), "S0": None}
    return x, gamma


def gamma_off(got, gamma, t):
    """The worst of |got - gamma| over its tolerance: t, and 2^-23 for each power of two below one (two roundings of the
    exponent); below 2^-60 anything up to 2^-60."""
    got = got.double()
    rel = t + 2.0 ** -23 * gamma.clamp(min=2.0 ** -60).log2().abs()
    return float(((got - gamma).abs() / (rel * gamma + 2.0 ** -60)).max())


@pytest.mark.parametrize("d", [64, 128])
def test_forward_decays_within_a_quarter(d):
    """Every Gamma_ts by itself.  Two exponentials of 2^-22, four fp32 roundings and P in two bf16 parts (each rounded by
    half a step: 2^-17 of its value at most)."""
    x, gamma = one_hot_tokens(96, d, 7)
    o, _ = efla.gated_fwd_chunked(**x, o_dtype=F32)
    assert gamma_off(o[0, :, :, :64].permute(1, 0, 2), gamma, 2.0 ** -17 + 2.0 ** -20) <= 1
    assert bool((o[..., 64:] == 0).all()) and efla.device_status() == 0


@pytest.mark.parametrize("d", [64, 128])
def test_backward_decays_within_a_quarter(d):
    """One entry of dO a head, (t, s): dg is Gamma_ts between s and t (no operand of it is split: two exponentials and four
    roundings), dbeta_s is Gamma_ts (through P, G and dY, each in two bf16 parts), and column s of dv is Gamma's row t (bf16)."""
    H = 288
    x, gamma = one_hot_tokens(H, d, 11)
    gen = torch.Generator().manual_seed(3)
    s = torch.randint(0, 54, (H,), generator=gen)
    s[::4] = 16 * torch.randint(0, 3, (len(s[::4]),), generator=gen) + 15  # a quarter's last token
    t = s + torch.randint(1, 10, (H,), generator=gen)
    h = torch.arange(H)
    want = gamma[h, t, s].cuda()
    dO = torch.zeros_like(x["v"])
    dO[0, t, h, s] = 1
    ws = efla.gated_fwd_chunked_train(**x)[2]
    got = efla.gated_bwd_chunked(*x.values(), dO, workspace=ws, saved=True)
    r = torch.arange(64, device="cuda")[:, None]
    s, t = s.cuda(), t.cuda()
    ref = torch.where((r > s) & (r <= t), want, 0.0)  # [64, H]
    assert gamma_off(got["dg"][0], ref, 2.0 ** -20) <= 1
    assert gamma_off(got["dbeta"][0], torch.where(r == s, want, 0.0), 3 * 2.0 ** -17 + 2.0 ** -19) <= 1
    dv = torch.zeros(64, H, d, device="cuda", dtype=torch.float64)
    dv[:, h.cuda(), s] = gamma[h, t.cpu()].cuda().t()  # (every token up to t is read by q_t)
    assert gamma_off(got["dv"][0], dv, 2.0 ** -8 + 3 * 2.0 ** -17 + 2.0 ** -19) <= 1
    assert efla.device_status() == 0


# ------------------------------------------------------------------------------ exact gate, tokens that write next to nothing
@pytest.mark.parametrize("dk, dv", [(128, 128), (64, 32)])
@pytest.mark.parametrize("size, beta", [(1e-10, 0.0), (1e-14, 1e-20), (1e-10, 1.0)])
def test_backward_exact_gate_of_vanishing_keys(dk, dv, size, beta):
    """beta lambda below the smallest fp32 number: alpha is beta, and its gradients are finite."""
    x = make(B=1, T=130, dk=dk, dv=dv, dtype=BF16, seed=3)
    x["k"][:, ::3] *= size
    x["beta"][:, ::2] = beta
    check_fwd(x, "exact")
    check_bwd(x, "exact")
    check_bwd(x)


# ------------------------------------------------------------------------------ saturated gates
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_prep_gradient_of_saturated_gates(dtype):
    """db = dbeta sigmoid(b) sigmoid(-b), relative to each value.  An exponential and a division within 2 steps of 2^-24, and
    four roundings."""
    b = torch.tensor([0.0, 0.5, 3.0, 9.0, 12.0, 15.0, 17.5, 30.0, 60.0, 80.0], device="cuda")
    b = torch.cat([b, -b])[None].to(dtype)  # one token, 20 heads
    gen = torch.Generator(device="cuda").manual_seed(1)
    q, dbeta = torch.ones(1, 1, 32, device="cuda", dtype=dtype), torch.randn(1, 20, generator=gen, device="cuda")
    A = torch.zeros(20, device="cuda")
    db = efla.gated_prep_bwd(q, q, b, b, A, A, q, q, dbeta, dbeta)["db"].double()
    ref = dbeta.double() * torch.sigmoid(b.double()) * torch.sigmoid(-b.double())
    t = 2.0 ** -20 + (2.0 ** -8 if dtype == BF16 else 0.0)
    assert bool(((db - ref).abs() <= t * ref.abs()).all()), (db / ref - 1).abs().max()


# ------------------------------------------------------------------------------ packed sequences around malformed bounds
@pytest.mark.parametrize("dtype, d", [(F32, 32), (BF16, 64), (BF16, 128)])
@pytest.mark.parametrize("bounds", [[0, 40, 200, 100], [-5, 10, 40, 100], [0, 70, 60, 60]])
def test_forward_packed_around_bad_bounds(dtype, d, bounds):
    """The sequences beside a malformed one are computed, and tokens of no sequence are left as they were."""
    x = make(B=1, T=100, N=3, dk=d, dv=d, dtype=dtype)
    cu = torch.tensor(bounds, dtype=torch.int32, device="cuda")
    S_T, o = torch.full((3, 4, d, d), 7.0, device="cuda"), torch.full((1, 100, 4, d), 7.0, device="cuda", dtype=dtype)
    efla.gated_fwd_chunked(**x, cu_seqlens=cu, o=o, S_T=S_T)
    assert efla.device_status() == 1
    free = torch.ones(100, dtype=torch.bool)
    for n, (a, b) in enumerate(zip(bounds, bounds[1:])):
        if 0 <= a <= b <= 100:
            free[a:b] = False
            ro, rS = gated.fwd(**{m: y[n:n + 1] if m == "S0" else y[:, a:b] for m, y in x.items()})
            close(o[:, a:b], ro, tol(dtype, d, d), f"o of sequence {n}")
            close(S_T[n:n + 1], rS, tol(dtype, d, d), f"S_T of sequence {n}")
        else:
            assert bool((S_T[n] == 7).all())
    assert bool((o[:, free] == 7).all())


# ------------------------------------------------------------------------------ rows that write nothing
@pytest.mark.parametrize("dtype, dk, dv", [(F32, 64, 64), (BF16, 128, 128), (BF16, 64, 32)])
@pytest.mark.parametrize("update", ["euler", "exact"])
def test_a_row_without_step_sizes_writes_nothing(dtype, dk, dv, update):
    """A padded batch row (beta = 0 for every token): no state, no outputs and no dv, not small ones; with a state and no
    decay, the state's bits.  The other row is as it is alone, and dbeta is the formula's."""
    x = make(B=2, T=150, dk=dk, dv=dv, dtype=dtype, S0=False)
    x["beta"][1] = 0
    x["beta"][0, ::3] = 0
    dO = torch.ones_like(x["v"])
    alone = {n: None if t is None else t[:1].contiguous() for n, t in x.items()}
    want_o, want_S = efla.gated_fwd_chunked(**alone, update=update)
    for call in (efla.gated_fwd_chunked, efla.gated_fwd_chunked_train):
        o, S = call(**x, update=update)[:2]
        assert not o[1].any() and not S[1].any()
        assert torch.equal(o[:1], want_o) and torch.equal(S[:1], want_S)
    got, ref = efla.gated_bwd_chunked(*x.values(), dO, update=update), gated.bwd(*x.values(), dO, None, update)
    assert not got["dv"][1].any() and not got["dv"][0, ::3].any()
    for n, r in ref.items():
        close(got[n][:1], r[:1], tol(dtype, dk, dv, True), n)
    close(got["dbeta"][1:], ref["dbeta"][1:], tol(dtype, dk, dv, True), "dbeta of the row")
    x["g"][1], x["S0"] = 0, torch.randn(2, 4, dk, dv, device="cuda")
    for call in (efla.gated_fwd_chunked, efla.gated_fwd_chunked_train):
        assert torch.equal(call(**x, update=update)[1][1], x["S0"][1])


def test_chunk_offsets_past_32_bits():
    """Forward, training forward and backward over more than 2^31 elements of q, k, v and o: the last row against the
    same call on it alone."""
    B, T, H, d = 64, 16400, 16, 128
    gen = torch.Generator(device="cuda").manual_seed(0)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda", dtype=BF16)  # noqa: E731
    q, v, dO = r(B, T, H, d) / 12, r(B, T, H, d), r(B, T, H, d)
    assert q.numel() > 2 ** 31
    g, beta = -r(B, T, H).float().abs(), torch.sigmoid(r(B, T, H).float())
    x, one = (q, q, v, g, beta), [t[-1:].contiguous() for t in (q, q, v, g, beta)]
    o, S, ws = efla.gated_fwd_chunked_train(*x)
    o1, S1, ws1 = efla.gated_fwd_chunked_train(*one)
    assert torch.equal(o[-1:], o1) and torch.equal(S[-1:], S1)
    got = efla.gated_bwd_chunked(*x, None, dO, workspace=ws, saved=True)
    want = efla.gated_bwd_chunked(*one, None, dO[-1:].contiguous(), workspace=ws1, saved=True)
    assert all(torch.equal(got[n][-1:], want[n]) for n in want)
    assert efla.device_status() == 0
