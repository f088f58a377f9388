"""Gated delta rule without a GPU: the 64-bit oracle against differences and its special cases, and
the refusals of the binding and of the C ABI (made before any launch)."""
import ctypes
import math

import pytest
import torch

import exact_delta_rule_gb300 as efla
import oracle
from oracle import gated


def inputs(B=2, T=5, Hk=1, H=2, dk=3, dv=4, seed=0):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=gen, dtype=torch.float64)  # noqa: E731
    return {"q": r(B, T, Hk, dk), "k": r(B, T, Hk, dk), "v": r(B, T, H, dv), "g": -r(B, T, H).abs(),
            "beta": torch.sigmoid(r(B, T, H)), "S0": r(B, H, dk, dv)}


@pytest.mark.parametrize("update", ["euler", "exact"])
def test_oracle_without_decay_is_the_delta_rule(update):
    x = inputs(Hk=2, H=2, dk=32, dv=32)
    x["g"].zero_()
    o, S = gated.fwd(**x, update=update)
    ref_o, ref_S = oracle.fwd(x["q"], x["k"], x["v"], x["beta"], x["S0"], update=update)
    torch.testing.assert_close(o, torch.as_tensor(ref_o).double(), rtol=0, atol=1e-9)
    torch.testing.assert_close(S, torch.as_tensor(ref_S).double(), rtol=0, atol=1e-9)


@pytest.mark.parametrize("update", ["euler", "exact"])
def test_oracle_gradients_are_the_differences(update):
    x = inputs()
    o, S = gated.fwd(**x, update=update)
    gen = torch.Generator().manual_seed(9)
    dO, dS = (torch.randn(t.shape, generator=gen, dtype=torch.float64) for t in (o, S))

    def loss(y):
        o, S = gated.fwd(**y, update=update)
        return float((o * dO).sum() + (S * dS).sum())

    grads = gated.bwd(x["q"], x["k"], x["v"], x["g"], x["beta"], x["S0"], dO, dS, update)
    h = 1e-6  # central differences: h^2 of the third derivative, 1e-16 / h of rounding
    for name, t in x.items():
        got = grads["d" + name]
        assert got.shape == t.shape
        for i in range(0, t.numel(), 3):
            up, down = t.clone(), t.clone()
            up.view(-1)[i] += h
            down.view(-1)[i] -= h
            diff = (loss({**x, name: up}) - loss({**x, name: down})) / (2 * h)
            assert math.isclose(diff, float(got.reshape(-1)[i]), rel_tol=1e-6, abs_tol=1e-7), (name, i)


def test_norm_oracles_against_autograd():
    gen = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(s, generator=gen, dtype=torch.float64, requires_grad=True)  # noqa: E731
    q, k, a, b, A, d = r(2, 3, 2, 8), r(2, 3, 2, 8), r(2, 3, 4), r(2, 3, 4), r(4), r(4)
    unit = lambda x: x / (x.square().sum(-1, keepdim=True) + 1e-6).sqrt()  # noqa: E731
    outs = [0.3 * unit(q), unit(k), -A.exp() * torch.nn.functional.softplus(a + d), torch.sigmoid(b)]
    ref = gated.prep(q, k, a, b, A, d, 0.3)
    for x, y in zip(outs, ref.values()):
        torch.testing.assert_close(x, y)
    dys = [torch.randn_like(x) for x in outs]
    want = torch.autograd.grad(outs, [q, k, a, b, A, d], dys)
    for x, y in zip(want, gated.prep_bwd(q, k, a, b, A, d, *dys, 0.3).values()):
        torch.testing.assert_close(x, y)
    o, z, w = r(2, 3, 8), r(2, 3, 8), r(8)
    y = torch.nn.functional.rms_norm(o, (8,), w, 1e-6) * torch.nn.functional.silu(z)
    torch.testing.assert_close(y, gated.norm_gate(o, z, w))
    dy = torch.randn_like(y)
    for x, u in zip(torch.autograd.grad(y, [o, z, w], dy), gated.norm_gate_bwd(o, z, w, dy).values()):
        torch.testing.assert_close(x, u)


# ------------------------------------------------------------------------------ refusals of the binding
def cpu_args(**over):
    x = {n: t.float() for n, t in inputs(B=2, T=4, Hk=2, H=4, dk=32, dv=32).items()} | over
    return [x[n] for n in ("q", "k", "v", "g", "beta")], x["S0"]


@pytest.mark.parametrize("over, what", [
    ({"q": torch.zeros(2, 4, 3, 32)}, "multiple"),
    ({"k": torch.zeros(2, 4, 2, 64)}, "k must be"),
    ({"v": torch.zeros(2, 5, 4, 32)}, "v must be"),
    ({"v": torch.zeros(2, 4, 4, 32, dtype=torch.bfloat16)}, "v must be"),
    ({"g": torch.zeros(2, 4, 4, dtype=torch.float64)}, "g must be"),
    ({"beta": torch.zeros(2, 4, 2)}, "beta must be"),
    ({"q": torch.zeros(2, 4, 2, 32, dtype=torch.float16)}, "bfloat16 or float32"),
    ({"q": torch.zeros(2, 2, 4, 32).transpose(1, 2)}, "q must be contiguous"),
    ({"S0": torch.zeros(2, 4, 32, 64)}, "S0 must be"),
    ({"S0": torch.zeros(2, 4, 32, 32, dtype=torch.bfloat16)}, "S0 must be"),
    ({}, "CUDA"),
])
def test_binding_refuses(over, what):
    args, S0 = cpu_args(**over)
    for call in (efla.gated_fwd_chunked, efla.gated_fwd_chunked_train):
        with pytest.raises(efla.EflaError, match=what):
            call(*args, S0)
    dO = torch.zeros_like(args[2])
    with pytest.raises(efla.EflaError):
        efla.gated_bwd_chunked(*args, S0, dO)
    with pytest.raises(efla.EflaError):
        efla.gated_decode_tokens(*args, torch.zeros(2, 4, 32, 32) if S0 is None else S0)


def test_a_stream_of_another_device_is_refused():
    from types import SimpleNamespace

    from exact_delta_rule_gb300 import gated as binding
    like = SimpleNamespace(get_device=lambda: 0, device="cuda:0")
    assert binding._stream(SimpleNamespace(device_index=0, cuda_stream=11), like) == 11
    with pytest.raises(efla.EflaError, match="the stream is on cuda:1"):
        binding._stream(SimpleNamespace(device_index=1, cuda_stream=11), like)
    with pytest.raises(efla.EflaError, match="CUDA tensors"):
        binding._on_device(torch.zeros(1))


def test_binding_refuses_more():
    args, S0 = cpu_args()
    with pytest.raises(efla.EflaError, match="unknown update"):
        efla.gated_fwd_chunked(*args, S0, update="implicit")
    with pytest.raises(efla.EflaError, match="cu_seqlens"):
        efla.gated_fwd_chunked(*args, None, torch.zeros(3, dtype=torch.int64))
    with pytest.raises(efla.EflaError, match="must be 1"):
        efla.gated_fwd_chunked(*args, None, torch.zeros(3, dtype=torch.int32))
    with pytest.raises(efla.EflaError, match="saved=True"):
        efla.gated_bwd_chunked(*args, S0, torch.zeros_like(args[2]), saved=True)
    with pytest.raises(efla.EflaError, match="dO must be"):
        efla.gated_bwd_chunked(*args, S0, torch.zeros_like(args[2]).bfloat16())
    with pytest.raises(efla.EflaError, match="o must be"):
        efla.gated_fwd_chunked(*args, S0, o_dtype=torch.float16)
    step = [x[:, 0].contiguous() for x in args]
    with pytest.raises(efla.EflaError, match="S must be"):
        efla.gated_decode_step(*step, torch.zeros(2, 4, 32, 32, dtype=torch.bfloat16))
    with pytest.raises(efla.EflaError, match="CUDA"):
        efla.gated_decode_step(*step, torch.zeros(2, 4, 32, 32))


def test_norm_bindings_refuse():
    q, a, p = torch.zeros(2, 3, 2, 32), torch.zeros(2, 3, 4), torch.zeros(4)
    with pytest.raises(efla.EflaError, match="a must be"):
        efla.gated_prep(q, q, a.double(), a, p, p)
    with pytest.raises(efla.EflaError, match="A_log must be"):
        efla.gated_prep(q, q, a, a, torch.zeros(3), p)
    with pytest.raises(efla.EflaError, match="q must be"):
        efla.gated_prep(q, q, a[0], a, p, p)
    with pytest.raises(efla.EflaError, match="CUDA"):
        efla.gated_prep(q, q, a, a, p, p)
    with pytest.raises(efla.EflaError, match="dg must be"):
        efla.gated_prep_bwd(q, q, a, a, p, p, q, q, a.bfloat16(), a)
    o, w = torch.zeros(2, 3, 64), torch.zeros(64)
    with pytest.raises(efla.EflaError, match="z must be"):
        efla.norm_gate(o, o[:1], w)
    with pytest.raises(efla.EflaError, match="w must be"):
        efla.norm_gate(o, o, w.bfloat16())
    with pytest.raises(efla.EflaError, match="dy must be"):
        efla.norm_gate_bwd(o, o, w, o.bfloat16())
    with pytest.raises(efla.EflaError, match="CUDA"):
        efla.norm_gate(o, o, w)


# ------------------------------------------------------------------------------ refusals of the C ABI
# Made-up device addresses that are never read: validation answers before any CUDA call.
A = [0x10000000 * (i + 1) for i in range(20)]


@pytest.fixture(scope="module")
def lib():
    return efla.gated._lib()


def c_fwd(lib, **kw):
    a = dict(q=A[0], k=A[1], v=A[2], g=A[3], beta=A[4], S0=None, cu=None, o=A[5], S_T=A[6], B=1, T=8, Hk=1, H=2, dk=64,
             dv=64, N=1, i=0, o_t=0, u=1, s=None) | kw
    return lib.efla_gated_fwd_chunked(*a.values())


@pytest.mark.parametrize("kw, code", [
    (dict(B=-1), 1), (dict(T=-1), 1), (dict(H=0), 1), (dict(Hk=0), 1), (dict(Hk=3, H=4), 1), (dict(dk=0), 1),
    (dict(dk=48), 2), (dict(dv=256), 2), (dict(i=2), 1), (dict(o_t=5), 1), (dict(u=2), 1), (dict(N=2), 1),
    (dict(cu=A[7], B=2, N=3), 1), (dict(q=None), 1), (dict(g=None), 1), (dict(beta=None), 1), (dict(o=None), 1),
    (dict(v=A[2] + 8), 1), (dict(g=A[3] + 4), 1), (dict(S_T=A[6] + 4), 1), (dict(o=A[0]), 1), (dict(S_T=A[3]), 1),
    (dict(S0=A[7], S_T=A[7] + 16), 1), (dict(T=1 << 30, H=4), 2), (dict(cu=A[7], N=-1), 1),
])
def test_c_forward_refuses(lib, kw, code):
    assert c_fwd(lib, **kw) == code, lib.efla_last_error()
    assert lib.efla_last_error()


def test_c_backward_refuses(lib):
    nb = ctypes.c_size_t(0)
    assert lib.efla_gated_bwd_workspace(1, 100, 1, 2, 64, 32, 0, ctypes.byref(nb)) == 0 and nb.value > 0
    assert lib.efla_gated_bwd_workspace(1, 100, 3, 4, 64, 32, 0, ctypes.byref(nb)) == 1

    def call(ws=A[14], size=1 << 40, **kw):
        a = dict(q=A[0], k=A[1], v=A[2], g=A[3], beta=A[4], S0=None, dO=A[5], dS_T=None, dq=A[6], dk=A[7], dv=A[8],
                 dg=A[9], dbeta=A[10], dS0=A[11], B=1, T=100, Hk=1, H=2, d=64, e=32, t=0, u=1, saved=0) | kw
        return lib.efla_gated_bwd_chunked(*a.values(), ws, size, None)

    assert call(ws=None) == 1 and call(size=16) == 1 and call(ws=A[14] + 8) == 1
    assert call(dq=None) == 1 and call(dO=None) == 1 and call(dq=A[1]) == 1 and call(dg=A[10]) == 1
    assert call(ws=A[2]) == 1 and call(Hk=3) == 1 and call(d=96) == 2
    train = dict(q=A[0], k=A[1], v=A[2], g=A[3], beta=A[4], S0=None, o=A[5], S_T=A[6], B=1, T=100, Hk=1, H=2, d=64, e=32,
                 t=0, u=1, ws=None, size=0, s=None)
    assert lib.efla_gated_fwd_chunked_train(*train.values()) == 1
    assert lib.efla_gated_fwd_chunked_train(*(train | dict(ws=A[0], size=1 << 40)).values()) == 1


def test_c_decode_and_norms_refuse(lib):
    step = dict(q=A[0], k=A[1], v=A[2], g=A[3], beta=A[4], S=A[5], o=A[6], B=2, Hk=1, H=2, dk=64, dv=64, i=0, o_t=0, u=1,
                s=None)
    for kw in (dict(S=None), dict(S=A[0]), dict(o=A[5]), dict(H=3, Hk=2), dict(dk=16), dict(g=None), dict(S=A[5] + 4)):
        assert lib.efla_gated_decode_step(*(step | kw).values()) in (1, 2), kw
    prep = dict(q=A[0], k=A[1], a=A[2], b=A[3], A=A[4], d=A[5], qo=A[6], ko=A[7], g=A[8], beta=A[9], n=4, Hk=1, H=2, dk=64,
                t=0, scale=1.0, eps=1e-6, s=None)
    for kw in (dict(n=-1), dict(Hk=0), dict(dk=100), dict(t=3), dict(scale=float("inf")), dict(eps=-1.0),
               dict(eps=float("nan")), dict(q=None), dict(qo=A[1]), dict(g=A[9]), dict(dk=0), dict(n=1 << 40)):
        assert lib.efla_gated_prep(*(prep | kw).values()) in (1, 2), kw
    norm = dict(o=A[0], z=A[1], w=A[2], y=A[3], rows=4, d=64, t=0, eps=1e-6, s=None)
    for kw in (dict(rows=-1), dict(d=80), dict(t=9), dict(eps=-1.0), dict(o=None), dict(w=A[2] + 4), dict(y=A[0] + 16),
               dict(y=A[2])):
        assert lib.efla_norm_gate(*(norm | kw).values()) in (1, 2), kw
    bwd = dict(o=A[0], z=A[1], w=A[2], dy=A[3], do=A[4], dz=A[5], dw=A[6], rows=4, d=64, t=0, eps=1e-6, ws=A[7], size=1 << 30,
               s=None)
    for kw in (dict(ws=None), dict(size=8), dict(do=A[0]), dict(dz=A[4]), dict(dw=None)):
        assert lib.efla_norm_gate_bwd(*(bwd | kw).values()) == 1, kw


def test_c_empty_calls_launch_nothing(lib):
    """Sizes of zero are valid and need no pointers."""
    assert c_fwd(lib, B=0, N=0, q=None, k=None, v=None, g=None, beta=None, o=None, S_T=None) == 0
    assert lib.efla_gated_decode_tokens(None, None, None, None, None, A[5], None, 2, 0, 1, 2, 64, 64, 0, 0, 1, None) == 0
    assert lib.efla_norm_gate(None, None, A[2], None, 0, 64, 0, 1e-6, None) == 0
    assert lib.efla_gated_prep(None, None, None, None, A[0], A[1], None, None, None, None, 0, 1, 2, 64, 0, 1.0, 1e-6,
                               None) == 0


# ------------------------------------------------------------------------------ which memory an output may share
def test_c_output_may_be_its_named_input_only(lib):
    """An output may be the one input that its contract names, not whatever else lies at that address.  (Refused calls
    only: an accepted one would launch.)"""
    prep = dict(q=A[0], k=A[1], a=A[2], b=A[3], A=A[4], d=A[5], qo=A[6], ko=A[7], g=A[8], beta=A[9], n=4, Hk=1, H=2, dk=64,
                t=0, scale=1.0, eps=1e-6, s=None)
    for kw in (dict(k=A[0], qo=A[0]),                  # rows of q overwritten while they are read as k
               dict(k=A[0], ko=A[0]),
               dict(k=A[0], qo=A[0], ko=A[0]),         # two outputs in one place
               dict(qo=A[6], ko=A[6]), dict(a=A[0], qo=A[0]), dict(A=A[0], qo=A[0])):
        assert lib.efla_gated_prep(*(prep | kw).values()) == 1, kw
        assert b"overlaps" in lib.efla_last_error()
    norm = dict(o=A[0], z=A[1], w=A[2], y=A[3], rows=4, d=64, t=0, eps=1e-6, s=None)
    for kw in (dict(w=A[0], y=A[0]), dict(w=A[1], y=A[1]), dict(z=A[0], w=A[0], y=A[0])):
        assert lib.efla_norm_gate(*(norm | kw).values()) == 1, kw
        assert b"overlaps" in lib.efla_last_error()
    for kw in (dict(S0=A[2], S_T=A[2]),                # the state over v
               dict(S0=A[4], S_T=A[4], beta=A[4]), dict(S0=A[6], S_T=A[6], cu=A[6])):
        assert c_fwd(lib, **kw) == 1, kw
        assert b"overlaps" in lib.efla_last_error()
    train = dict(q=A[0], k=A[1], v=A[2], g=A[3], beta=A[4], S0=A[2], o=A[5], S_T=A[2], B=1, T=8, Hk=1, H=2, d=64, e=64,
                 t=0, u=1, ws=A[10], size=1 << 40, s=None)
    assert lib.efla_gated_fwd_chunked_train(*train.values()) == 1
    assert b"overlaps" in lib.efla_last_error()


@pytest.mark.parametrize("B, T, H", [((1 << 31) - 1, 0, (1 << 31) - 1), ((1 << 31) - 1,) * 3, (1 << 21, 1 << 21, 1 << 22)])
def test_c_sizes_whose_product_passes_64_bits(lib, B, T, H):
    """Refused, not wrapped around to a size that looks small."""
    nb = ctypes.c_size_t(0)
    assert lib.efla_gated_bwd_workspace(B, T, 1, H, 64, 64, 0, ctypes.byref(nb)) == 2
    assert b"token-heads" in lib.efla_last_error()


def test_binding_refuses_sizes_past_32_bits():
    """A size that ctypes would cut to its low 32 bits is refused, not taken for a small one (tensors without memory)."""
    z = lambda *s, dtype=torch.bfloat16: torch.empty(s, dtype=dtype, device="meta")  # noqa: E731
    d, f = 2 ** 32 + 32, torch.float32
    with pytest.raises(efla.EflaError, match="2147483647"):
        efla.norm_gate(z(1, d), z(1, d), z(d, dtype=f))
    with pytest.raises(efla.EflaError, match="2147483647"):
        efla.norm_gate_bwd(z(1, d), z(1, d), z(d, dtype=f), z(1, d))
    for dk, H in ((d, 4), (32, 2 ** 32 + 4)):
        q, a, p = z(1, 1, dk), z(1, H), z(H, dtype=f)
        with pytest.raises(efla.EflaError, match="2147483647"):
            efla.gated_prep(q, q, a, a, p, p)
    for dk, dv in ((d, 32), (32, d)):
        q, v, g = z(1, 1, 1, dk), z(1, 1, 1, dv), z(1, 1, 1, dtype=f)
        with pytest.raises(efla.EflaError, match="2147483647"):
            efla.gated_fwd_chunked(q, q, v, g, g, return_state=False)
    for i in range(6):
        sizes = [1, 64, 1, 1, 32, 32]
        sizes[i] += 2 ** 32
        with pytest.raises(efla.EflaError, match="2147483647"):
            efla.gated_bwd_workspace(*sizes, torch.bfloat16)
