"""Short convolution, selective scan and group norm without a GPU: the 64-bit oracle against autograd of another form,
and the refusals of the binding and of the C ABI (made before any launch)."""
import ctypes

import pytest
import torch

import exact_delta_rule_gb300 as efla
from oracle import ssm


def rand(gen, *shape, grad=False):
    return torch.randn(shape, generator=gen, dtype=torch.float64, requires_grad=grad)


@pytest.mark.parametrize("W, T", [(2, 5), (3, 1), (4, 2), (4, 9)])
@pytest.mark.parametrize("silu", [True, False])
def test_oracle_convolution(W, T, silu):
    gen = torch.Generator().manual_seed(W + T)
    x, w, bias, s0 = (rand(gen, *s, grad=True) for s in ((2, T, 3), (3, W), (3,), (2, W - 1, 3)))
    full = torch.cat([s0, x], 1)
    s = torch.nn.functional.conv1d(full.transpose(1, 2), w[:, None], bias, groups=3).transpose(1, 2)
    y, end = torch.nn.functional.silu(s) if silu else s, full[:, T:]
    for a, b in zip((y, end), ssm.conv(x, w, bias, s0, silu)):
        torch.testing.assert_close(a.detach(), b)
    dy, dend = torch.randn_like(y), torch.randn_like(end)
    want = torch.autograd.grad([y, end], [x, w, bias, s0], [dy, dend])
    got = ssm.conv_bwd(x, w, bias, s0, dy, dend, silu)
    for a, name in zip(want, ("dx", "dw", "dbias", "dstate0")):
        torch.testing.assert_close(a, got[name])
        assert bool((ssm.conv_bwd(x, w, bias, s0, dy, dend, silu, size=True)[name] >= a.abs() - 1e-12).all())


@pytest.mark.parametrize("G, gate", [(1, True), (2, False)])
def test_oracle_scan_in_closed_form(G, gate):
    """h_T = sum_s e^{A (delta_{s+1} + .. + delta_T)} delta_s x_s B_s, by autograd of that sum."""
    gen = torch.Generator().manual_seed(G)
    B, T, D, N = 2, 6, 4, 3
    x, dt, A_log, Bm, Cm, Dk, bias, z, S0 = (rand(gen, *s, grad=True) for s in (
        (B, T, D), (B, T, D), (D, N), (B, T, G, N), (B, T, G, N), (D,), (D,), (B, T, D), (B, D, N)))
    delta = torch.nn.functional.softplus(dt + bias)
    run = delta.cumsum(1)
    A = -A_log.exp()
    each = torch.arange(D) // (D // G)
    states = []
    for t in range(T):
        h = torch.exp(A * run[:, t, :, None]) * S0
        for s in range(t + 1):
            h = h + torch.exp(A * (run[:, t] - run[:, s])[..., None]) * (delta[:, s] * x[:, s])[..., None] * Bm[:, s, each]
        states.append(h)
    y = torch.stack([(h * Cm[:, t, each]).sum(-1) for t, h in enumerate(states)], 1) + Dk * x
    if gate:
        y = y * torch.nn.functional.silu(z)
    zz = z if gate else None
    for a, b in zip((y, states[-1]), ssm.scan(x, dt, A_log, Bm, Cm, Dk, bias, zz, S0)):
        torch.testing.assert_close(a.detach(), b)
    dy, dS = torch.randn_like(y), torch.randn_like(S0)
    names = ["x", "dt", "A_log", "B", "C", "D", "dt_bias", "S0"] + ["z"] * gate
    want = torch.autograd.grad([y, states[-1]], [x, dt, A_log, Bm, Cm, Dk, bias, S0] + [z] * gate, [dy, dS])
    got = ssm.scan_bwd(x, dt, A_log, Bm, Cm, Dk, bias, zz, S0, dy, dS)
    large = ssm.scan_bwd(x, dt, A_log, Bm, Cm, Dk, bias, zz, S0, dy, dS, size=True)
    for a, name in zip(want, names):
        torch.testing.assert_close(a, got["d" + name])
        assert bool((large["d" + name] >= a.abs() - 1e-12).all()), name


def test_oracle_scan_gradients_are_the_differences():
    gen = torch.Generator().manual_seed(3)
    names = ("x", "dt", "A_log", "B", "C", "D", "dt_bias", "z", "S0")
    a = dict(zip(names, (rand(gen, *s) for s in ((1, 4, 2), (1, 4, 2), (2, 3), (1, 4, 1, 3), (1, 4, 1, 3), (2,), (2,), (1, 4, 2),
                                                 (1, 2, 3)))))
    y, S = ssm.scan(*a.values())
    dy, dS = torch.randn_like(y), torch.randn_like(S)

    def loss(v):
        y, S = ssm.scan(*v.values())
        return float((y * dy).sum() + (S * dS).sum())

    got = ssm.scan_bwd(*a.values(), dy, dS)
    h = 1e-6  # central differences: h^2 of the third derivative, 1e-16 / h of rounding
    for name, t in a.items():
        for i in range(t.numel()):
            up, down = t.clone(), t.clone()
            up.view(-1)[i] += h
            down.view(-1)[i] -= h
            diff = (loss({**a, name: up}) - loss({**a, name: down})) / (2 * h)
            assert abs(diff - float(got["d" + name].reshape(-1)[i])) <= 1e-6 * (1 + abs(diff)), (name, i)


@pytest.mark.parametrize("shape, groups", [((3, 12), 4), ((2, 5, 6), 2), ((2, 2, 3, 4), 1)])
@pytest.mark.parametrize("silu", [True, False])
def test_oracle_group_norm(shape, groups, silu):
    gen = torch.Generator().manual_seed(groups)
    x, w, b = rand(gen, *shape, grad=True), rand(gen, shape[-1], grad=True), rand(gen, shape[-1], grad=True)
    s = torch.nn.functional.group_norm(x.movedim(-1, 1), groups, w, b, 1e-5).movedim(1, -1)
    y = torch.nn.functional.silu(s) if silu else s
    torch.testing.assert_close(y.detach(), ssm.group_norm(x, w, b, groups, silu=silu)[0])
    dy = torch.randn_like(y)
    got, sizes = ssm.group_norm_bwd(x, w, b, groups, dy, silu=silu)
    for a, name in zip(torch.autograd.grad(y, [x, w, b], dy), ("dx", "dw", "db")):
        torch.testing.assert_close(a, got[name])
        assert bool((sizes[name] >= a.abs() - 1e-12).all())


# ------------------------------------------------------------------------------ refusals of the binding
def conv_args(**over):
    a = {"x": torch.zeros(2, 5, 16), "w": torch.zeros(16, 4), "bias": torch.zeros(16), "state0": torch.zeros(2, 3, 16)} | over
    return a


@pytest.mark.parametrize("over, what", [
    ({"x": torch.zeros(2, 5, 16, dtype=torch.float16)}, "bfloat16 or float32"),
    ({"x": torch.zeros(5, 16)}, "x must be"),
    ({"x": torch.zeros(2, 16, 5).transpose(1, 2)}, "x must be contiguous"),
    ({"w": torch.zeros(16, 4, dtype=torch.bfloat16)}, "w must be"),
    ({"w": torch.zeros(8, 4)}, "w must be"),
    ({"w": torch.zeros(16)}, "w must be"),
    ({"bias": torch.zeros(4)}, "bias must be"),
    ({"state0": torch.zeros(2, 4, 16)}, "state0 must be"),
    ({"state0": torch.zeros(2, 3, 16, dtype=torch.bfloat16)}, "state0 must be"),
    ({}, "CUDA"),
])
def test_convolution_refuses(over, what):
    a = conv_args(**over)
    with pytest.raises(efla.EflaError, match=what):
        efla.causal_conv(**a)
    with pytest.raises(efla.EflaError):
        efla.causal_conv_bwd(**a, dy=torch.zeros(2, 5, 16))
    with pytest.raises(efla.EflaError):
        efla.causal_conv_step(a["x"][:, 0], a["w"], a["bias"], a["state0"])


def test_convolution_refuses_more():
    a = conv_args()
    with pytest.raises(efla.EflaError, match="activation"):
        efla.causal_conv(**a, activation="gelu")
    with pytest.raises(efla.EflaError, match="cu_seqlens"):
        efla.causal_conv(a["x"][:1], a["w"], cu_seqlens=torch.zeros(3, dtype=torch.int64))
    with pytest.raises(efla.EflaError, match="must be 1"):
        efla.causal_conv(a["x"], a["w"], cu_seqlens=torch.zeros(3, dtype=torch.int32))
    with pytest.raises(efla.EflaError, match="dy must be"):
        efla.causal_conv_bwd(**a, dy=torch.zeros(2, 4, 16))
    with pytest.raises(efla.EflaError, match="state must be"):
        efla.causal_conv_step(torch.zeros(2, 16), a["w"], None, torch.zeros(2, 2, 16))


def scan_args(**over):
    return {"x": torch.zeros(2, 5, 16), "dt": torch.zeros(2, 5, 16), "A_log": torch.zeros(16, 32), "B": torch.zeros(2, 5, 2, 32),
            "C": torch.zeros(2, 5, 2, 32), "D": torch.zeros(16), "dt_bias": torch.zeros(16), "z": torch.zeros(2, 5, 16),
            "S0": torch.zeros(2, 16, 32)} | over


@pytest.mark.parametrize("over, what", [
    ({"x": torch.zeros(2, 5, 16, dtype=torch.float64)}, "bfloat16 or float32"),
    ({"x": torch.zeros(2, 16, 5).transpose(1, 2)}, "x must be contiguous"),
    ({"dt": torch.zeros(2, 5, 8)}, "dt must be"),
    ({"dt": torch.zeros(2, 5, 16, dtype=torch.bfloat16)}, "dt must be"),
    ({"A_log": torch.zeros(16)}, "A_log must be"),
    ({"A_log": torch.zeros(8, 32)}, "A_log must be"),
    ({"B": torch.zeros(2, 5, 32)}, "B 4-D"),
    ({"B": torch.zeros(2, 5, 2, 16)}, "B must be"),
    ({"C": torch.zeros(2, 5, 1, 32)}, "C must be"),
    ({"D": torch.zeros(16, dtype=torch.bfloat16)}, "D must be"),
    ({"dt_bias": torch.zeros(2)}, "dt_bias must be"),
    ({"z": torch.zeros(2, 5, 32)}, "z must be"),
    ({"S0": torch.zeros(2, 32, 16)}, "S0 must be"),
    ({}, "CUDA"),
])
def test_scan_refuses(over, what):
    a = scan_args(**over)
    for call in (efla.ssm_scan, efla.ssm_scan_train):
        with pytest.raises(efla.EflaError, match=what):
            call(**a)
    with pytest.raises(efla.EflaError):
        efla.ssm_scan_bwd(**a, dy=torch.zeros(2, 5, 16))


def test_scan_refuses_more():
    a = scan_args()
    with pytest.raises(efla.EflaError, match="saved=True"):
        efla.ssm_scan_bwd(**a, dy=torch.zeros(2, 5, 16), saved=True)
    with pytest.raises(efla.EflaError, match="dy must be"):
        efla.ssm_scan_bwd(**a, dy=torch.zeros(2, 5, 16).bfloat16())
    with pytest.raises(efla.EflaError, match="dS_T must be"):
        efla.ssm_scan_bwd(**a, dy=torch.zeros(2, 5, 16), dS_T=torch.zeros(2, 16, 16))
    one = {k: v[:, 0].contiguous() if k in ("x", "dt", "B", "C", "z") else v for k, v in a.items() if k != "S0"}
    with pytest.raises(efla.EflaError, match="S must be"):
        efla.ssm_step(**one, S=torch.zeros(2, 16, 32, dtype=torch.bfloat16))
    with pytest.raises(efla.EflaError, match="CUDA"):
        efla.ssm_step(**one, S=torch.zeros(2, 16, 32))
    with pytest.raises(efla.EflaError, match="exceeds"):
        efla.ssm_scan_workspace(1, 1 << 32, 16, 16)


def test_group_norm_refuses():
    x, w = torch.zeros(3, 5, 16), torch.zeros(16)
    for over, what in (({"x": torch.zeros(16)}, "x must be"), ({"x": x.half()}, "bfloat16 or float32"), ({"groups": 3}, "multiple of"),
                       ({"groups": 0}, "multiple of"), ({"w": torch.zeros(8)}, "w must be"), ({"b": w.bfloat16()}, "b must be"),
                       ({"x": torch.zeros(3, 16, 5).transpose(1, 2)}, "x must be contiguous"), ({}, "CUDA")):
        a = {"x": x, "w": w, "b": w, "groups": 4} | over
        with pytest.raises(efla.EflaError, match=what):
            efla.group_norm(**a)
        with pytest.raises(efla.EflaError):
            efla.group_norm_bwd(**a, stats=torch.zeros(3, 4, 2), dy=x)
    with pytest.raises(efla.EflaError, match="activation"):
        efla.group_norm(x, w, w, 4, activation="relu")
    with pytest.raises(efla.EflaError, match="stats must be"):
        efla.group_norm_bwd(x, w, w, 4, torch.zeros(3, 4), x)
    with pytest.raises(efla.EflaError, match="dy must be"):
        efla.group_norm_bwd(x, w, w, 4, torch.zeros(3, 4, 2), x.bfloat16())


# ------------------------------------------------------------------------------ refusals of the C ABI
# Made-up device addresses that are never read: validation answers before any CUDA call.
A = [0x100000000 * (i + 1) for i in range(24)]


@pytest.fixture(scope="module")
def lib():
    return efla.ssm._lib()


def c_conv(lib, **kw):
    a = dict(x=A[0], w=A[1], bias=A[2], s0=A[3], cu=None, y=A[4], sT=A[5], B=2, T=8, D=64, W=4, N=2, dt=0, act=1, s=None) | kw
    return lib.efla_causal_conv(*a.values())


@pytest.mark.parametrize("kw, code", [
    (dict(B=-1), 1), (dict(T=-1), 1), (dict(D=0), 1), (dict(D=12), 2), (dict(W=1), 2), (dict(W=5), 2), (dict(dt=2), 1),
    (dict(act=2), 1), (dict(N=3), 1), (dict(cu=A[6]), 1), (dict(B=1, cu=A[6], N=-1), 1), (dict(x=None), 1), (dict(w=None), 1),
    (dict(y=None), 1), (dict(x=A[0] + 8), 1), (dict(bias=A[2] + 4), 1), (dict(y=A[0]), 1), (dict(sT=A[3]), 1),
    (dict(B=1 << 20, T=1 << 20, N=1 << 20), 2), (dict(D=1 << 21), 2),
])
def test_c_convolution_refuses(lib, kw, code):
    assert c_conv(lib, **kw) == code, lib.efla_last_error()
    assert lib.efla_last_error()


def test_c_convolution_backward_and_step_refuse(lib):
    n = ctypes.c_size_t()
    assert lib.efla_causal_conv_bwd_workspace(2, 8, 64, 4, None) == 1
    assert lib.efla_causal_conv_bwd_workspace(2, 8, 60, 4, ctypes.byref(n)) == 2
    assert lib.efla_causal_conv_bwd_workspace(2, 8, 64, 4, ctypes.byref(n)) == 0 and n.value >= 64 * 5 * 4

    def bwd(**kw):
        a = dict(x=A[0], w=A[1], bias=A[2], s0=None, dy=A[3], dT=None, dx=A[4], dw=A[5], db=A[6], d0=None, B=2, T=8, D=64, W=4,
                 dt=0, act=1, ws=A[7], wb=n.value, s=None) | kw
        return lib.efla_causal_conv_bwd(*a.values())

    for kw in (dict(wb=n.value - 1), dict(ws=None), dict(ws=A[0]), dict(dx=A[0]), dict(dw=A[1]), dict(dy=None), dict(dw=None),
               dict(act=7), dict(dx=A[4] + 2)):
        assert bwd(**kw) == 1, kw
    assert bwd(W=8) == 2

    def step(**kw):
        a = dict(x=A[0], w=A[1], bias=None, st=A[2], y=A[3], B=2, D=64, W=4, dt=0, act=1, s=None) | kw
        return lib.efla_causal_conv_step(*a.values())

    for kw in (dict(st=None), dict(y=A[0]), dict(st=A[0]), dict(B=-1), dict(y=A[3] + 8)):
        assert step(**kw) == 1, kw
    assert step(D=4) == 2
    assert step(B=0, x=None, st=None, y=None) == 0


def c_scan(lib, **kw):
    a = dict(x=A[0], dt=A[1], A=A[2], B=A[3], C=A[4], D=A[5], bias=A[6], z=A[7], S0=A[8], cu=None, y=A[9], S_T=A[10], rows=2, T=8,
             ch=64, N=16, G=1, seqs=2, type=0, ws=A[11], wb=1 << 28, s=None) | kw
    return lib.efla_ssm_scan(*a.values())


@pytest.mark.parametrize("kw, code", [
    (dict(rows=-1), 1), (dict(T=-1), 1), (dict(ch=0), 1), (dict(ch=60), 2), (dict(N=8), 2), (dict(N=256), 2), (dict(G=0), 1),
    (dict(G=3), 1), (dict(ch=24, G=2), 2), (dict(type=3), 1), (dict(seqs=1), 1), (dict(cu=A[12]), 1), (dict(x=None), 1),
    (dict(dt=None), 1), (dict(A=None), 1), (dict(B=None), 1), (dict(C=None), 1), (dict(y=None), 1), (dict(z=A[7] + 8), 1),
    (dict(y=A[0]), 1), (dict(S_T=A[9]), 1), (dict(S_T=A[8] + 16), 1), (dict(T=4096, ws=None), 1), (dict(T=4096, wb=16), 1),
    (dict(T=4096, ws=A[0]), 1), (dict(rows=1 << 16, seqs=1 << 16, T=1 << 16), 2),
])
def test_c_scan_refuses(lib, kw, code):
    assert c_scan(lib, **kw) == code, lib.efla_last_error()
    assert lib.efla_last_error()


def test_c_scan_training_and_step_refuse(lib):
    n = ctypes.c_size_t()
    assert lib.efla_ssm_bwd_workspace(2, 100, 64, 16, 1, None) == 1
    assert lib.efla_ssm_bwd_workspace(2, 100, 64, 24, 1, ctypes.byref(n)) == 2
    assert lib.efla_ssm_scan_workspace(2, 100, 64, 16, 1, 3, 0, ctypes.byref(n)) == 1
    assert lib.efla_ssm_bwd_workspace(2, 100, 64, 16, 1, ctypes.byref(n)) == 0

    def train(**kw):
        a = dict(x=A[0], dt=A[1], A=A[2], B=A[3], C=A[4], D=None, bias=None, z=A[5], S0=None, y=A[6], S_T=A[7], rows=2, T=100, ch=64,
                 N=16, G=1, type=0, ws=A[8], wb=n.value, s=None) | kw
        return lib.efla_ssm_scan_train(*a.values())

    for kw in (dict(ws=None), dict(wb=n.value - 1), dict(ws=A[0]), dict(y=A[5]), dict(type=9), dict(C=None)):
        assert train(**kw) == 1, kw

    def bwd(**kw):
        a = dict(x=A[0], dt=A[1], A=A[2], B=A[3], C=A[4], D=A[5], bias=A[6], z=A[7], S0=None, dy=A[8], dS_T=None, dx=A[9], ddt=A[10],
                 dA=A[11], dB=A[12], dC=A[13], dD=A[14], db=A[15], dz=A[16], dS0=A[17], rows=2, T=100, ch=64, N=16, G=1, type=0,
                 saved=1, ws=A[18], wb=n.value, s=None) | kw
        return lib.efla_ssm_scan_bwd(*a.values())

    for kw in (dict(ws=None), dict(wb=n.value - 1), dict(ws=A[9]), dict(dz=None), dict(z=None), dict(dx=A[0]), dict(dB=None),
               dict(dA=None), dict(dS0=A[9] + 16), dict(dy=None), dict(G=0)):
        assert bwd(**kw) == 1, kw

    def step(**kw):
        a = dict(x=A[0], dt=A[1], A=A[2], B=A[3], C=A[4], D=None, bias=None, z=None, S=A[5], y=A[6], rows=2, ch=64, N=16, G=1, type=0,
                 s=None) | kw
        return lib.efla_ssm_step(*a.values())

    for kw in (dict(S=None), dict(S=A[0]), dict(y=A[5]), dict(rows=-1), dict(G=5)):
        assert step(**kw) == 1, kw
    assert step(N=4) == 2
    assert step(rows=0, x=None, dt=None, B=None, C=None, S=None, y=None) == 0


def test_c_group_norm_refuses(lib):
    n = ctypes.c_size_t()
    assert lib.efla_group_norm_workspace(2, 9, 64, 4, 0, 1, None) == 1
    assert lib.efla_group_norm_workspace(2, 9, 60, 4, 0, 1, ctypes.byref(n)) == 2
    assert lib.efla_group_norm_workspace(2, 1, 64, 4, 0, 0, ctypes.byref(n)) == 0 and n.value == 0
    assert lib.efla_group_norm_workspace(2, 9, 64, 4, 0, 1, ctypes.byref(n)) == 0

    def fwd(**kw):
        a = dict(x=A[0], w=A[1], b=A[2], y=A[3], stats=A[4], rows=2, L=9, C=64, groups=4, dt=0, act=1, eps=1e-5, ws=A[5], wb=n.value,
                 s=None) | kw
        return lib.efla_group_norm(*a.values())

    for kw in (dict(rows=-1), dict(L=-1), dict(C=0), dict(groups=0), dict(groups=5), dict(dt=2), dict(act=-1), dict(eps=-1.0),
               dict(eps=float("nan")), dict(x=None), dict(y=None), dict(w=A[1] + 4), dict(y=A[0] + 16), dict(stats=A[0]),
               dict(L=30000, wb=1 << 28, ws=A[3]), dict(L=30000, wb=16), dict(L=30000, ws=None)):
        assert fwd(**kw) == 1, kw
    assert fwd(rows=0, x=None, y=None) == 0

    def bwd(**kw):
        a = dict(x=A[0], w=A[1], b=A[2], stats=A[3], dy=A[4], dx=A[5], dw=A[6], db=A[7], rows=2, L=9, C=64, groups=4, dt=0, act=1,
                 ws=A[8], wb=n.value, s=None) | kw
        return lib.efla_group_norm_bwd(*a.values())

    for kw in (dict(stats=None), dict(dy=None), dict(dx=None), dict(ws=None), dict(wb=n.value - 1), dict(dx=A[0]), dict(dw=A[1])):
        assert bwd(**kw) == 1, kw


def test_workspaces_of_whole_and_cut_rows():
    assert efla.ssm_scan_workspace(64, 2048, 2048, 16) == 0      # rows enough to fill the GPU
    assert efla.ssm_scan_workspace(1, 8, 2048, 16) == 0          # nothing to cut
    one = efla.ssm_scan_workspace(1, 8192, 2048, 16)
    assert one > 0 and efla.ssm_scan_workspace(1, 8192, 2048, 16, N=1) >= one
    assert efla.ssm_bwd_workspace(0, 8, 64, 16) >= 0

def test_workspaces_of_the_longest_rows():
    """Rows up to the accepted length: the number of segments, and with it the workspace, goes on smoothly."""
    longest = 2 ** 31 - 1 - 4096
    for D, N in ((8, 16), (64, 128)):
        for packed in (None, 1, 3):
            if packed:
                a, b = (efla.ssm_scan_workspace(1, T, D, N, N=packed) for T in (longest, longest - 20_000_000))
            else:
                a, b = (efla.ssm_scan_workspace(1, T, D, N) for T in (longest, longest - 20_000_000))
            assert 0 < a < 1 << 32 and abs(a - b) <= 0.1 * b, (D, N, packed, a, b)
        a, b = (efla.ssm_bwd_workspace(1, T, D, N) for T in (longest, longest - 20_000_000))
        assert b < a < 1.02 * b, (D, N, a, b)
    assert 0 < efla.ssm._bytes("efla_causal_conv_bwd_workspace", 1, longest, 8, 4) < 1 << 32
