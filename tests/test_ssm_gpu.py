"""Short convolution, selective scan and group norm on the GPU against the 64-bit oracle (oracle/ssm.py).

An output is a sum of products in fp32.  Its tolerance is a share of the sum of the magnitudes of what it is made of
(the oracle with size=True) plus, for bf16 outputs, half a step: 2^-8 of the value.  The share:
  convolution   W + 2 roundings of 2^-24 before the activation and a sigmoid of 2 + 1.2 |s| ulp (|s| < 8: 7e-7) with
                three more roundings; a sum over n tokens n roundings.
  scan          the state is carried by T factors e^{A delta}, each off by 1.5e-7 of itself (the exponential
                instruction) and 2^-24 from a multiplication and an addition; softplus and the exponent's product are
                1e-6 of delta (|dt| < 12), of which e^{-v} v <= 0.4 reaches a product of any number of factors with
                exponent v; the sum over N entries and the gate are 20 roundings more.  A gradient goes through two
                such chains, and a sum over all tokens adds as many roundings.
"""
import math

import pytest
import torch

import exact_delta_rule_gb300 as efla
from oracle import ssm

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


def close(got, ref, size, share, what=""):
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    if not ref.numel():
        return
    step = 2.0 ** -8 if got.dtype == BF16 else 0.0
    got = got.double()
    assert bool(torch.isfinite(got).all()), f"{what}: non-finite values"
    over = (got - ref).abs() - step * ref.abs() - share * size
    i = int(over.argmax())
    assert float(over.max()) <= 1e-30, \
        f"{what}: {float(got.flatten()[i])} for {float(ref.flatten()[i])} (size {float(size.flatten()[i])}), share {share:.1e}, over by {float(over.max()):.2e}"


def randn(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda")


# ------------------------------------------------------------------------------------ convolution
def conv_inputs(B=2, T=37, D=40, W=4, dtype=F32, bias=True, state=True, N=None, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return {"x": randn(gen, B, T, D).to(dtype), "w": randn(gen, D, W), "bias": randn(gen, D) if bias else None,
            "state0": randn(gen, B if N is None else N, W - 1, D).to(dtype) if state else None}


def conv_share(W, n=1):
    return (W + 2 + 3 + n) * U + 7e-7


def check_conv(a, silu):
    act = "silu" if silu else None
    y, end = efla.causal_conv(**a, activation=act)
    ref, ref_end = ssm.conv(**a, silu=silu)
    size, _ = ssm.conv(**a, silu=silu, size=True)
    close(y, ref, size, conv_share(a["w"].shape[1]), "y")
    assert torch.equal(end.double(), ref_end)
    return y, end


@pytest.mark.parametrize("T", [0, 1, 2, 3, 4, 15, 16, 17, 300])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_convolution_lengths(dtype, W, T):
    check_conv(conv_inputs(T=T, W=W, dtype=dtype, seed=T), silu=T % 2 == 0)


@pytest.mark.parametrize("B, T, D", [(1, 1, 8), (3, 70, 8), (300, 1, 24), (1, 5000, 16), (2, 33, 1000), (1, 40, 6144), (0, 5, 16)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_convolution_shapes(dtype, B, T, D):
    check_conv(conv_inputs(B=B, T=T, D=D, dtype=dtype, bias=D != 24, state=T != 70), silu=True)
    a = conv_inputs(B=B, T=T, D=D, dtype=dtype)
    y, none = efla.causal_conv(**a, return_state=False)
    assert none is None and torch.equal(y, efla.causal_conv(**a)[0])


def cu_of(lens):
    return torch.tensor([0] + list(lens), dtype=torch.int32).cumsum(0).to(torch.int32).cuda()


LENS = [5, 0, 16, 1, 2, 130, 0, 3, 63, 200, 4]


@pytest.mark.parametrize("W", [2, 4])
@pytest.mark.parametrize("state", [True, False])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D, lens", [(72, LENS), (8, [40] * 100), (8, [1] * 300 + [500, 3]), (1000, [17] * 30)])
def test_convolution_packed(dtype, W, state, D, lens):
    a = conv_inputs(B=1, T=sum(lens), D=D, W=W, dtype=dtype, state=state, N=len(lens))
    y, end = efla.causal_conv(**a, cu_seqlens=cu_of(lens))
    at = 0
    for i, n in enumerate(lens):
        one = {**a, "x": a["x"][:, at:at + n].contiguous(), "state0": a["state0"][i:i + 1].contiguous() if state else None}
        y1, end1 = efla.causal_conv(**one)
        assert torch.equal(y[:, at:at + n], y1) and torch.equal(end[i:i + 1], end1), i
        at += n
    assert efla.device_status() == 0


@pytest.mark.parametrize("call", ["conv", "scan"])
@pytest.mark.parametrize("bounds, good", [([0, 40, 200, 100], [0]), ([-5, 10, 40, 100], [1, 2]), ([0, 70, 60, 60], [0, 2]),
                                          ([10, 20, 20, 90], [0, 1, 2])])
def test_packed_around_bad_bounds(call, bounds, good):
    """Well-formed sequences (empty ones too) are computed, the others' states and tokens of no sequence left alone."""
    cu = torch.tensor(bounds, dtype=torch.int32, device="cuda")
    if call == "conv":
        a = conv_inputs(B=1, T=100, D=16, N=3)
        y, end = torch.full((1, 100, 16), 7.0, device="cuda"), torch.full((3, 3, 16), 7.0, device="cuda")
        efla.causal_conv(**a, cu_seqlens=cu, y=y, state_T=end)
    else:
        a = scan_inputs(B=1, T=100, D=16, seqs=3)
        y, end = torch.full((1, 100, 16), 7.0, device="cuda"), torch.full((3, 16, 16), 7.0, device="cuda")
        efla.ssm_scan(**a, cu_seqlens=cu, y=y, S_T=end)
    assert efla.device_status() == (1 if len(good) < 3 else 0)
    mine = torch.zeros(100, dtype=torch.bool, device="cuda")
    for n in range(3):
        if n not in good:
            assert bool((end[n] == 7).all())
            continue
        lo, hi = bounds[n:n + 2]
        mine[lo:hi] = True
        one = {k: v[:, lo:hi].contiguous() if k in ("x", "dt", "B", "C", "z") and v is not None else v for k, v in a.items()}
        state = "state0" if call == "conv" else "S0"
        one[state] = a[state][n:n + 1].contiguous()
        y1, end1 = efla.causal_conv(**one) if call == "conv" else efla.ssm_scan(**one)
        assert torch.equal(y[:, lo:hi], y1) and torch.equal(end[n:n + 1], end1)
    assert bool((y[0, ~mine] == 7).all())


@pytest.mark.parametrize("T", [0, 1, 2, 3, 5, 31, 32, 35, 200])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_convolution_backward(dtype, W, T):
    check_conv_bwd(conv_inputs(T=T, W=W, dtype=dtype, seed=T, state=T % 2 == 1, bias=T != 5), silu=T != 2)


@pytest.mark.parametrize("B, T, D", [(1, 1, 8), (70, 3, 8), (2, 700, 16), (5, 90, 264), (1, 50, 6144), (0, 4, 16)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_convolution_backward_shapes(dtype, B, T, D):
    check_conv_bwd(conv_inputs(B=B, T=T, D=D, dtype=dtype), silu=True)


@pytest.mark.parametrize("B, T, D", [(500, 20, 2048), (36, 250, 6144), (1, 9001, 512)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_convolution_backward_fills_the_gpu(dtype, B, T, D):
    """Several tiles of runs a CTA, and runs longer than the ring of copies."""
    check_conv_bwd(conv_inputs(B=B, T=T, D=D, dtype=dtype), silu=True)


def check_conv_bwd(a, silu):
    gen = torch.Generator(device="cuda").manual_seed(5)
    B, T, D = a["x"].shape
    W = a["w"].shape[1]
    dy, dend = randn(gen, B, T, D).to(a["x"].dtype), randn(gen, B, W - 1, D).to(a["x"].dtype)
    if T == 3:
        dend = None
    got = efla.causal_conv_bwd(**a, dy=dy, dstate_T=dend, activation="silu" if silu else None)
    ref = ssm.conv_bwd(**a, dy=dy, dstate_T=dend, silu=silu)
    size = ssm.conv_bwd(**a, dy=dy, dstate_T=dend, silu=silu, size=True)
    for name, r in ref.items():
        if r is None:
            assert got[name] is None
            continue
        n = B * T if name in ("dw", "dbias") else W
        close(got[name], r, size[name], 2 * conv_share(W, n), name)
    again = efla.causal_conv_bwd(**a, dy=dy, dstate_T=dend, activation="silu" if silu else None, need_dstate0=False)
    assert again["dstate0"] is None
    for name, v in again.items():
        assert v is None or torch.equal(v, got[name]), name  # a fixed order of addition


@pytest.mark.parametrize("B, D", [(1, 8), (3, 40), (257, 136)])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_convolution_step_continues_the_prompt(dtype, W, B, D):
    a = conv_inputs(B=B, T=6, D=D, W=W, dtype=dtype)
    y, end = efla.causal_conv(**a)
    state = a["state0"].clone()
    steps = [efla.causal_conv_step(a["x"][:, t].contiguous(), a["w"], a["bias"], state) for t in range(6)]
    assert torch.equal(state, end)
    ref, _ = ssm.conv(**a)
    size, _ = ssm.conv(**a, size=True)
    close(torch.stack(steps, 1), ref, size, conv_share(W), "steps")


# ------------------------------------------------------------------------------------ scan
def scan_inputs(B=2, T=37, D=40, N=16, G=1, dtype=F32, z=True, skip=True, bias=True, S0=True, seqs=None, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: randn(gen, *s)  # noqa: E731
    return {"x": r(B, T, D).to(dtype), "dt": r(B, T, D).to(dtype), "A_log": r(D, N), "B": r(B, T, G, N).to(dtype),
            "C": r(B, T, G, N).to(dtype), "D": r(D) if skip else None, "dt_bias": r(D) - 2 if bias else None,
            "z": r(B, T, D).to(dtype) if z else None, "S0": r(B if seqs is None else seqs, D, N) if S0 else None}


def scan_share(T, links=1, n=0):
    return links * (T * (1.5e-7 + 2 * U) + 1e-6 + 20 * U) + n * U


def check_scan(a, **kw):
    y, S = efla.ssm_scan(**a, **kw)
    ref, ref_S = ssm.scan(**a)
    size, size_S = ssm.scan(**a, size=True)
    share = scan_share(a["x"].shape[1])
    close(y, ref, size, share, "y")
    close(S, ref_S, size_S, share, "S_T")
    assert efla.device_status() == 0
    return y, S


@pytest.mark.parametrize("T", [0, 1, 2, 15, 16, 17, 31, 33, 127, 128, 300])
@pytest.mark.parametrize("dtype, N", [(F32, 16), (BF16, 16), (F32, 64), (BF16, 128)])
def test_scan_lengths(dtype, N, T):
    check_scan(scan_inputs(T=T, N=N, dtype=dtype, seed=T))


@pytest.mark.parametrize("B, D, G", [(1, 8, 1), (3, 136, 1), (1, 128, 2), (2, 272, 2), (1, 96, 4), (0, 16, 1)])
@pytest.mark.parametrize("N", [16, 32, 64, 128])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_scan_shapes(dtype, N, B, D, G):
    check_scan(scan_inputs(B=B, T=50, D=D, N=N, G=G, dtype=dtype, z=D != 136, skip=D != 272, bias=G != 4, S0=B != 1))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_scan_options(dtype):
    a = scan_inputs(T=200, dtype=dtype)
    y, S = check_scan(a)
    y2, none = efla.ssm_scan(**a, return_state=False)
    assert none is None and torch.equal(y, y2)
    inplace = {**a, "S0": a["S0"].clone()}  # S0 and S_T the same memory
    y2, S2 = efla.ssm_scan(**inplace, S_T=inplace["S0"])
    assert torch.equal(y2, y) and torch.equal(S2, S) and S2.data_ptr() == inplace["S0"].data_ptr()


@pytest.mark.parametrize("N", [16, 128])
@pytest.mark.parametrize("state", [True, False])
@pytest.mark.parametrize("lens", [LENS, [700], [0, 0], [1, 1000, 0, 77], [1] * 300])
def test_scan_packed(N, state, lens):
    a = scan_inputs(B=1, T=sum(lens), D=24, N=N, seqs=len(lens), S0=state)
    y, S = efla.ssm_scan(**a, cu_seqlens=cu_of(lens))
    at = 0
    for i, n in enumerate(lens[:20]):
        one = {k: v[:, at:at + n].contiguous() if k in ("x", "dt", "B", "C", "z") else v for k, v in a.items()}
        one["S0"] = a["S0"][i:i + 1].contiguous() if state else None
        ref, ref_S = ssm.scan(**one)
        size, size_S = ssm.scan(**one, size=True)
        close(y[:, at:at + n], ref, size, scan_share(n), f"y {i}")
        close(S[i:i + 1], ref_S, size_S, scan_share(n), f"S {i}")
        at += n
    assert efla.device_status() == 0


@pytest.mark.parametrize("what", ["still", "fast", "masked", "frozen", "large dt", "no input"])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_scan_extremes(dtype, what):
    a = scan_inputs(T=150, D=24, N=32, dtype=dtype)
    if what == "still":
        a["A_log"].fill_(-30.0)            # hardly any decay: a sum over all tokens
    elif what == "fast":
        a["A_log"].fill_(6.0)              # forgets at once
    elif what == "masked":
        a["dt"][:, 40:].fill_(-math.inf)   # a padded row: the state stays
    elif what == "frozen":
        a["dt"].fill_(-200.0)
    elif what == "large dt":
        a["dt"].fill_(30.0)
        a["A_log"].fill_(-5.0)
    elif what == "no input":
        a["x"].zero_()
    # (e^{A delta} of a delta of 30 has an exponent up to 0.2 a token)
    check_scan(a)
    if what == "masked":  # bit for bit (rows as short as these are not cut, so both add in the same order)
        S40, S100 = (efla.ssm_scan(**{k: v[:, :n].contiguous() if k in ("x", "dt", "B", "C", "z") else v for k, v in a.items()})[1]
                     for n in (40, 100))
        assert torch.equal(S40, S100)


def test_scan_keeps_bad_values_in_their_row():
    a = scan_inputs(B=3, T=60, D=16)
    y, S = efla.ssm_scan(**a)
    a["x"][1, 20, 3] = math.nan
    a["B"][2, 30, 0, 1] = math.inf
    y2, S2 = efla.ssm_scan(**a)
    assert torch.equal(y2[0], y[0]) and torch.equal(S2[0], S[0])
    assert torch.equal(y2[1, :20], y[1, :20]) and torch.equal(y2[2, :30], y[2, :30])
    others = [c for c in range(16) if c != 3]
    assert torch.equal(y2[1][:, others], y[1][:, others]) and bool(y2[1, 20:, 3].isnan().all())


def test_scan_groups_of_four_channels():
    a = scan_inputs(T=50, D=24, G=2, N=64)
    check_scan(a)
    check_scan_bwd(a)
    with pytest.raises(efla.EflaError, match="multiple of 8"):
        efla.ssm_scan(**scan_inputs(T=50, D=24, G=2, dtype=BF16))


def check_scan_bwd(a, saved=True, dS=True):
    gen = torch.Generator(device="cuda").manual_seed(7)
    B, T, D = a["x"].shape
    dy = randn(gen, B, T, D).to(a["x"].dtype)
    dS_T = randn(gen, B, D, a["A_log"].shape[1]) if dS else None
    y, S, ws = efla.ssm_scan_train(**a)
    ref, ref_S = ssm.scan(**a)
    size, size_S = ssm.scan(**a, size=True)
    close(y, ref, size, scan_share(T), "y")
    close(S, ref_S, size_S, scan_share(T), "S_T")
    got = efla.ssm_scan_bwd(**a, dy=dy, dS_T=dS_T, workspace=ws if saved else None, saved=saved)
    ref = ssm.scan_bwd(**a, dy=dy, dS_T=dS_T)
    size = ssm.scan_bwd(**a, dy=dy, dS_T=dS_T, size=True)
    for name, r in ref.items():
        if r is None:
            assert got[name] is None
            continue
        n = {"dA_log": B * T, "dD": B * T, "ddt_bias": B * T, "dB": D, "dC": D}.get(name, 0)
        close(got[name], r, size[name], scan_share(T, 2, n), name)
    assert efla.device_status() == 0
    return got, dy, dS_T


@pytest.mark.parametrize("T", [0, 1, 2, 4, 15, 16, 17, 33, 64, 130, 300])
@pytest.mark.parametrize("dtype, N", [(F32, 16), (BF16, 16), (F32, 64), (BF16, 128)])
def test_scan_backward_lengths(dtype, N, T):
    check_scan_bwd(scan_inputs(T=T, N=N, dtype=dtype, seed=T), saved=T != 33, dS=T != 17)


@pytest.mark.parametrize("B, D, G", [(1, 8, 1), (3, 136, 1), (1, 128, 2), (2, 272, 2), (1, 96, 4), (0, 16, 1)])
@pytest.mark.parametrize("N", [16, 32, 64, 128])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_scan_backward_shapes(dtype, N, B, D, G):
    check_scan_bwd(scan_inputs(B=B, T=50, D=D, N=N, G=G, dtype=dtype, z=D != 136, skip=D != 272, bias=G != 4, S0=B != 1))


def test_scan_backward_repeats_bit_for_bit():
    a = scan_inputs(B=2, T=400, D=264, dtype=BF16)
    got, dy, dS = check_scan_bwd(a)
    for saved in (True, False):
        ws = efla.ssm_scan_train(**a)[2] if saved else None
        again = efla.ssm_scan_bwd(**a, dy=dy, dS_T=dS, workspace=ws, saved=saved)
        for name, v in again.items():
            assert torch.equal(v, got[name]), name
    assert efla.ssm_scan_bwd(**a, dy=dy, need_dS0=False)["dS0"] is None


@pytest.mark.parametrize("what", ["still", "fast", "masked"])
def test_scan_backward_extremes(what):
    a = scan_inputs(T=100, D=24, N=32)
    if what == "masked":
        a["dt"][:, 40:].fill_(-math.inf)
    else:
        a["A_log"].fill_(-30.0 if what == "still" else 6.0)
    check_scan_bwd(a)


@pytest.mark.parametrize("B, D, G", [(1, 8, 1), (3, 136, 1), (2, 272, 2), (7, 96, 4), (600, 40, 1)])
@pytest.mark.parametrize("N", [16, 32, 64, 128])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_step_continues_the_prompt(dtype, N, B, D, G):
    a = scan_inputs(B=B, T=3, D=D, N=N, G=G, dtype=dtype, z=D != 136, skip=D != 272, bias=G != 4)
    S = a["S0"].clone()
    ys = []
    for t in range(3):
        tok = {k: v[:, t].contiguous() if k in ("x", "dt", "B", "C", "z") and v is not None else v for k, v in a.items() if k != "S0"}
        ys.append(efla.ssm_step(**tok, S=S))
    ref, ref_S = ssm.scan(**a)
    size, size_S = ssm.scan(**a, size=True)
    close(torch.stack(ys, 1), ref, size, scan_share(3), "y")
    close(S, ref_S, size_S, scan_share(3), "S")


# ------------------------------------------------------------------------------------ group norm
def norm_share(L):
    return (L + 610) * U + 7e-7


def check_group_norm(shape, groups, dtype, silu, affine=True, offset=0.0, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    C = shape[-1]
    x = (randn(gen, *shape) * (0.5 + torch.rand(C, generator=gen, device="cuda")) + randn(gen, C) + offset).to(dtype)
    w, b = (randn(gen, C), randn(gen, C)) if affine else (None, None)
    dy, act = randn(gen, *shape).to(dtype), "silu" if silu else None
    L = math.prod(shape[1:-1])
    y, stats = efla.group_norm(x, w, b, groups, activation=act, return_stats=True)
    assert torch.equal(y, efla.group_norm(x, w, b, groups, activation=act))
    same = x.clone()
    assert torch.equal(efla.group_norm(same, w, b, groups, activation=act, y=same), y)
    if not x.numel():
        assert efla.group_norm_bwd(x, w, b, groups, stats, dy, activation=act)["dw"].abs().sum() == 0
        return
    ref, ref_stats = ssm.group_norm(x, w, b, groups, silu=silu)
    mean, r = ref_stats.unbind(-1)
    width = (mean.abs() + 1 / r)  # the size of a group's values
    share = norm_share(L)
    close(stats[..., 0], mean, width, share, "mean")
    close(stats[..., 1], r, r * width * r, 2 * share, "r")
    spread = (width * r).reshape(shape[0], *[1] * (len(shape) - 2), groups).repeat_interleave(C // groups, -1)
    n = ssm.group_norm(x, None, None, groups)[0].abs() + spread
    size = n * (w.abs() if affine else 1) + (b.abs() if affine else 0)
    close(y, ref, 1.1 * size, 4 * share, "y")
    got = efla.group_norm_bwd(x, w, b, groups, stats, dy, activation=act)
    ref, size = ssm.group_norm_bwd(x, w, b, groups, dy, silu=silu)
    big = float(spread.max()) ** 2  # what an error of the mean or r, relative to the values' size, does to n
    for name, v in ref.items():
        if v is None:
            assert got[name] is None
            continue
        close(got[name], v, size[name] * (1 + big), 4 * share + (0 if name == "dx" else x.numel() // C * U), name)
    again = efla.group_norm_bwd(x, w, b, groups, stats, dy, activation=act)
    for name, v in again.items():
        assert v is None or torch.equal(v, got[name]), name


@pytest.mark.parametrize("shape, groups", [
    ((1, 8), 1), ((7, 2048), 16), ((1000, 256), 1), ((33, 64), 8), ((5, 24), 3), ((3, 40), 1), ((2, 96), 32), ((65, 640), 16),
    ((9, 4096), 2), ((2, 8192), 1), ((700, 16), 16), ((0, 16), 2), ((3, 192), 4), ((513, 264), 11),
    ((700, 1000), 8), ((9, 5000), 40), ((3, 8192), 8192), ((650, 24), 24), ((2, 30000), 3)])
@pytest.mark.parametrize("dtype, silu", [(F32, True), (BF16, False)])
def test_group_norm_of_tokens(dtype, silu, shape, groups):
    check_group_norm(shape, groups, dtype, silu)


@pytest.mark.parametrize("shape, groups", [
    ((2, 2, 8), 8), ((1, 9, 320), 32), ((3, 5, 7, 40), 4), ((2, 1000, 64), 2), ((1, 64, 64, 320), 32), ((40, 3, 16), 1),
    ((2, 0, 16), 2), ((1, 300, 1032), 3), ((200, 17, 8), 4),
    ((700, 5, 48), 16), ((2, 4099, 24), 24), ((1, 70001, 8), 1), ((3, 33, 2056), 1), ((1, 5000, 520), 5),
    ((2, 30000, 64), 2)])
@pytest.mark.parametrize("dtype, silu", [(F32, True), (BF16, True), (BF16, False)])
def test_group_norm_of_maps(dtype, silu, shape, groups):
    check_group_norm(shape, groups, dtype, silu)


@pytest.mark.parametrize("shape, groups", [
    ((5, 2048), 1), ((1, 1040), 2), ((901, 1032), 1), ((3, 4104), 3), ((2, 8192), 1), ((40, 16384), 2), ((3, 8200), 1),
    ((700, 16, 256), 8), ((9, 100, 768), 12), ((5, 64, 512), 32), ((1, 5, 7, 240), 5), ((2, 511, 32), 2), ((610, 2, 4096), 1)])
@pytest.mark.parametrize("dtype, silu", [(F32, True), (BF16, True), (BF16, False)])
def test_group_norm_of_groups_a_team_holds(dtype, silu, shape, groups):
    check_group_norm(shape, groups, dtype, silu)


def test_group_norm_keeps_a_bad_parameter_in_its_group():
    for shape, groups in [((33, 520), 13), ((33, 2080), 2), ((9, 20, 520), 5)]:
        x, dy = torch.randn(shape, device="cuda"), torch.randn(shape, device="cuda")
        w, b = torch.randn(shape[-1], device="cuda"), torch.randn(shape[-1], device="cuda")
        y, stats = efla.group_norm(x, w, b, groups, activation="silu", return_stats=True)
        good = efla.group_norm_bwd(x, w, b, groups, stats, dy, activation="silu")
        b[0] = math.nan
        y2 = efla.group_norm(x, w, b, groups, activation="silu")
        bad = efla.group_norm_bwd(x, w, b, groups, stats, dy, activation="silu")
        each = shape[-1] // groups
        assert torch.equal(y2[..., 1:], y[..., 1:])
        assert torch.equal(bad["dx"][..., each:], good["dx"][..., each:])


@pytest.mark.parametrize("shape, groups", [((20, 512), 4), ((2, 300, 64), 4)])
def test_group_norm_extremes(shape, groups):
    check_group_norm(shape, groups, F32, True, affine=False)
    check_group_norm(shape, groups, F32, False, offset=300.0)  # a mean far from 0
    y = efla.group_norm(torch.full(shape, 3.0, device="cuda"), None, torch.ones(shape[-1], device="cuda"), groups)
    assert bool((y == 1).all())  # no variance: n = 0
    x = torch.randn(shape, device="cuda")
    y = efla.group_norm(x, None, None, groups)
    x[1, ..., 0] = math.nan
    y2 = efla.group_norm(x, None, None, groups)
    each = shape[-1] // groups
    assert bool(y2[1, ..., :each].isnan().all()) and torch.equal(y2[0], y[0]) and torch.equal(y2[1, ..., each:], y[1, ..., each:])


# ------------------------------------------------------------------------------------ the manner of the calls
def between_sentinels(t, pad=4096):
    """A copy of t in the middle of a larger allocation filled with a pattern, and a check of the rest."""
    n = t.numel() * t.element_size()
    room = torch.full((n + 2 * pad,), 0x5a, dtype=torch.uint8, device="cuda")
    room[pad:pad + n] = t.contiguous().view(-1).view(torch.uint8)
    view = room[pad:pad + n].view(t.dtype).view(t.shape)
    return view, lambda: bool((room[:pad] == 0x5a).all()) and bool((room[pad + n:] == 0x5a).all())


@pytest.mark.parametrize("dtype, N, D, T", [(BF16, 16, 136, 77), (F32, 64, 24, 200), (BF16, 128, 40, 5)])
def test_calls_write_only_their_outputs(dtype, N, D, T):
    a = scan_inputs(T=T, D=D, N=N, dtype=dtype)
    inputs = {k: v.clone() for k, v in a.items()}
    y, ok_y = between_sentinels(torch.zeros_like(a["x"]))
    S, ok_S = between_sentinels(torch.zeros_like(a["S0"]))
    ws, ok_ws = between_sentinels(torch.zeros(max(16, efla.ssm_bwd_workspace(2, T, D, N)), dtype=torch.uint8, device="cuda"))
    y0, S0, _ = efla.ssm_scan_train(**a, workspace=ws, y=y, S_T=S)
    assert ok_y() and ok_S() and ok_ws()
    efla.ssm_scan_bwd(**a, dy=a["z"], workspace=ws, saved=True)
    assert ok_ws()
    assert torch.equal(y, efla.ssm_scan(**a)[0])
    for k, v in a.items():
        assert torch.equal(v, inputs[k]), k
    c = conv_inputs(T=T, D=D, dtype=dtype)
    y, ok_y = between_sentinels(torch.zeros_like(c["x"]))
    end, ok_end = between_sentinels(torch.zeros_like(c["state0"]))
    efla.causal_conv(**c, y=y, state_T=end)
    assert ok_y() and ok_end() and torch.equal(y, efla.causal_conv(**c)[0])


def test_streams_and_graphs():
    a, c = scan_inputs(B=1, T=900, D=128, dtype=BF16, S0=False), conv_inputs(B=1, T=900, D=128, dtype=BF16)
    dy = a["z"].clone()

    def everything(stream=None):
        y, _ = efla.causal_conv(**c, stream=stream)
        out, S, ws = efla.ssm_scan_train(**a, stream=stream)
        g = efla.ssm_scan_bwd(**a, dy=dy, workspace=ws, saved=True, stream=stream)
        gc = efla.causal_conv_bwd(**c, dy=dy, stream=stream)
        y2, S2 = efla.ssm_scan(**a, stream=stream)
        heads, st = efla.group_norm(out[0], a["D"], a["dt_bias"], 4, return_stats=True, stream=stream)
        whole, st2 = efla.group_norm(out, None, None, 4, activation="silu", return_stats=True, stream=stream)
        gn = efla.group_norm_bwd(out, None, None, 4, st2, dy, activation="silu", stream=stream)
        gh = efla.group_norm_bwd(out[0], a["D"], a["dt_bias"], 4, st, dy[0], stream=stream)
        return [y, out, S, y2, S2, heads, st, whole, st2, gn["dx"], *gh.values(), *g.values(), *(v for v in gc.values() if v is not None)]

    want = everything()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = everything(side)
    side.synchronize()
    for x, y in zip(want, got):
        assert torch.equal(x, y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = everything()
    for _ in range(2):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(want, got):
            assert torch.equal(x, y)
    a["x"].mul_(-1)  # a replay reads the inputs anew: from a state of 0 the scan is odd in x
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[1], -want[1])


def test_two_calls_at_once():
    """Two streams, a workspace each, give what one after the other does."""
    a = [scan_inputs(B=1, T=2000, D=64, dtype=BF16, seed=s) for s in (1, 2)]
    want = [efla.ssm_scan(**x) for x in a]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in a]
    got = []
    for _ in range(3):
        got += [efla.ssm_scan(**x, stream=s) for x, s in zip(a, streams)]
    torch.cuda.synchronize()
    for i, (y, S) in enumerate(got):
        assert torch.equal(y, want[i % 2][0]) and torch.equal(S, want[i % 2][1])


def test_offsets_past_32_bits():
    """2^31 elements and more of a row: the last tokens against the same tokens continued from a state."""
    B, T, D, N = 1, 131200, 16384, 16
    gen = torch.Generator(device="cuda").manual_seed(0)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda", dtype=BF16)  # noqa: E731
    a = {"x": r(B, T, D), "dt": r(B, T, D), "A_log": torch.full((D, N), 1.0, device="cuda"), "B": r(B, T, 1, N), "C": r(B, T, 1, N)}
    y, S = efla.ssm_scan(**a)
    tail = {k: v[:, -400:].contiguous() if k != "A_log" else v for k, v in a.items()}
    y2, S2 = efla.ssm_scan(**tail)  # (e^{-2.7 delta} of a delta of 0.8: nothing from 200 tokens before is left)
    assert torch.equal(y[:, -100:], y2[:, -100:]) and torch.equal(S, S2)
    w = torch.randn(D, 4, device="cuda")
    y, end = efla.causal_conv(a["x"], w)
    y2, end2 = efla.causal_conv(tail["x"], w)
    assert torch.equal(y[:, -100:], y2[:, -100:]) and torch.equal(end, end2)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_a_layer_trains_and_decodes(dtype):
    """Convolution, projections and scan as a layer runs them: a prompt, its gradients against the oracle's chain on the
    same intermediate values, and a token after the prompt against the prompt extended by it."""
    gen = torch.Generator(device="cuda").manual_seed(4)
    B, T, D, N = 2, 45, 64, 16
    x, w, bias = randn(gen, B, T + 1, D).to(dtype), randn(gen, D, 4) / 2, randn(gen, D) / 2
    proj = (randn(gen, D, D + 2 * N) / 8).to(dtype)
    A_log, Dk, dtb, z = torch.log(torch.rand(D, N, device="cuda") * 4 + 0.5), randn(gen, D), randn(gen, D) - 2, randn(gen, B, T + 1, D).to(dtype)

    def parts(u):
        p = u @ proj
        lead = u.shape[:-1]
        return p[..., :D].contiguous(), p[..., D:D + N].reshape(*lead, 1, N).contiguous(), p[..., D + N:].reshape(*lead, 1, N).contiguous()

    u, cstate = efla.causal_conv(x[:, :T].contiguous(), w, bias)
    dt, Bm, Cm = parts(u)
    zz = z[:, :T].contiguous()
    y, S, ws = efla.ssm_scan_train(u, dt, A_log, Bm, Cm, Dk, dtb, zz)
    dy = randn(gen, B, T, D).to(dtype)
    g = efla.ssm_scan_bwd(u, dt, A_log, Bm, Cm, Dk, dtb, zz, None, dy, workspace=ws, saved=True)
    back = torch.cat([g["ddt"], g["dB"].flatten(2), g["dC"].flatten(2)], -1)
    du = (g["dx"].float() + back.float() @ proj.float().T).to(dtype)
    gx = efla.causal_conv_bwd(x[:, :T].contiguous(), w, bias, None, du)
    args = (u, dt, A_log, Bm, Cm, Dk, dtb, zz, None)
    ref, size = (ssm.scan_bwd(*args, dy, size=s) for s in (False, True))
    for name in ("dx", "ddt", "dB", "dC", "dz", "dA_log", "dD", "ddt_bias"):
        close(g[name], ref[name], size[name], scan_share(T, 2, B * T + D), name)
    cargs = (x[:, :T], w, bias, None, du)
    ref, size = (ssm.conv_bwd(*cargs, size=s) for s in (False, True))
    for name in ("dx", "dw", "dbias"):
        close(gx[name], ref[name], size[name], 2 * conv_share(4, B * T), name)
    # one more token
    u1 = efla.causal_conv_step(x[:, T].contiguous(), w, bias, cstate)
    dt1, B1, C1 = parts(u1)
    S1 = S.clone()
    y1 = efla.ssm_step(u1, dt1, A_log, B1, C1, Dk, dtb, z[:, T].contiguous(), S1)
    one = [t.unsqueeze(1) for t in (u1, dt1)] + [A_log] + [t.unsqueeze(1) for t in (B1, C1)] + [Dk, dtb, z[:, T:], S]
    ref, ref_S = ssm.scan(*one)
    size, size_S = ssm.scan(*one, size=True)
    close(y1.unsqueeze(1), ref, size, scan_share(1), "token")
    close(S1, ref_S, size_S, scan_share(1), "state")
    full, _ = efla.causal_conv(x, w, bias)
    ref, _ = ssm.conv(x, w, bias)
    csize, _ = ssm.conv(x, w, bias, size=True)
    close(u1, ref[:, T], csize[:, T], conv_share(4), "convolved token")


def test_convolution_feeds_the_gated_delta_rule():
    """q, k and v of a gated delta mixer behind their convolution: prompt and following token give the same as one prompt."""
    gen = torch.Generator(device="cuda").manual_seed(6)
    B, T, H, d = 2, 40, 2, 64
    qkv, w = randn(gen, B, T + 1, 3 * H * d), randn(gen, 3 * H * d, 4) / 2
    a, b, A_log, dtb = randn(gen, B, T + 1, H), randn(gen, B, T + 1, H), randn(gen, H), randn(gen, H)

    def mixer(c, at):
        lead = c.shape[:-1]
        q, k, v = (t.reshape(*lead, H, d).contiguous() for t in c.split(H * d, -1))
        p = efla.gated_prep(q, k, a[:, at].contiguous(), b[:, at].contiguous(), A_log, dtb)
        return p["q"], p["k"], v, p["g"], p["beta"]

    c, state = efla.causal_conv(qkv[:, :T].contiguous(), w)
    _, S = efla.gated_fwd_chunked(*mixer(c, slice(0, T)))
    o = efla.gated_decode_step(*mixer(efla.causal_conv_step(qkv[:, T].contiguous(), w, None, state), T), S)
    whole, _ = efla.causal_conv(qkv, w)
    ref, _ = efla.gated_fwd_chunked(*mixer(whole, slice(0, T + 1)))
    # two orders of the same fp32 sums: 2 x 2 (d + 64) roundings of the largest output
    assert float((o - ref[:, T]).abs().max()) <= 8 * (d + 64) * U * float(ref.abs().max())
