"""Short convolution, selective scan and group norm at the ends of what their contract allows, on the GPU: decays that no
float holds, runs and rows of the largest sizes, groups whose first value or mean is far from the others."""
import math

import pytest
import torch

import exact_delta_rule_gb300 as efla
from norm_bounds import check_gradients, check_stats, check_y, far_values
from oracle import ssm
from test_ssm_gpu import BF16, F32, between_sentinels, check_scan, check_scan_bwd, close, cu_of, scan_inputs, scan_share

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------------------------ scan: decays out of range
def steep(T, D=24, N=32, padded=5, seqs=None, **kw):
    """A_log at and past the largest whose exponential an fp32 number holds, beside ordinary ones; the last tokens masked."""
    a = scan_inputs(T=T, D=D, N=N, seqs=seqs, **kw)
    for i, v in enumerate((88.2, 88.5, 89.0, 95.0, 700.0)):
        a["A_log"][i::7, i::3] = v
    if padded:
        a["dt"][:, -padded:] = -math.inf
    return a


@pytest.mark.parametrize("T", [1, 2, 6, 7, 37, 130])
@pytest.mark.parametrize("dtype, N", [(F32, 16), (BF16, 32), (F32, 128)])
def test_scan_of_steep_decays(dtype, N, T):
    """Tokens of delta = 0 (a row that ends inside a group of four, a masked one) keep the state, whatever the decay."""
    check_scan(steep(T, N=N, dtype=dtype, padded=0))
    y, S = check_scan(steep(T + 5, N=N, dtype=dtype))
    assert bool(torch.isfinite(S).all())


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_scan_of_steep_decays_in_cut_rows(dtype):
    a = steep(1500, B=1, N=16, dtype=dtype, padded=700)  # whole segments of masked tokens
    assert efla.ssm_scan_workspace(1, 1500, 24, 16) > 0
    check_scan(a)
    lens = [3, 0, 700, 1, 90, 706]
    a = steep(1500, B=1, N=16, dtype=dtype, padded=300, seqs=len(lens))
    y, S = efla.ssm_scan(**a, cu_seqlens=cu_of(lens))
    at = 0
    for i, n in enumerate(lens):
        one = {k: v[:, at:at + n].contiguous() if k in ("x", "dt", "B", "C", "z") else v for k, v in a.items()}
        one["S0"] = a["S0"][i:i + 1].contiguous()
        ref, ref_S = ssm.scan(**one)
        size, size_S = ssm.scan(**one, size=True)
        close(y[:, at:at + n], ref, size, scan_share(n), f"y {i}")
        close(S[i:i + 1], ref_S, size_S, scan_share(n), f"S {i}")
        at += n


@pytest.mark.parametrize("T, padded", [(6, 5), (37, 0), (37, 9), (900, 300)])
@pytest.mark.parametrize("dtype, N", [(F32, 16), (BF16, 32), (F32, 128)])
def test_scan_gradients_of_steep_decays(dtype, N, T, padded):
    got, _, _ = check_scan_bwd(steep(T, N=N, dtype=dtype, padded=padded))
    if padded:
        assert bool((got["ddt"][:, -padded:] == 0).all())


@pytest.mark.parametrize("B", [1, 600])
@pytest.mark.parametrize("dtype, N", [(F32, 16), (BF16, 128)])
def test_step_of_steep_decays(dtype, N, B):
    a = steep(1, B=B, N=N, dtype=dtype, padded=0)
    a["dt"][::2] = -math.inf
    S = a["S0"].clone()
    tok = {k: v[:, 0].contiguous() if k in ("x", "dt", "B", "C", "z") else v for k, v in a.items() if k != "S0"}
    y = efla.ssm_step(**tok, S=S)
    ref, ref_S = ssm.scan(**a)
    size, size_S = ssm.scan(**a, size=True)
    close(y.unsqueeze(1), ref, size, scan_share(1), "y")
    close(S, ref_S, size_S, scan_share(1), "S")
    assert torch.equal(S[::2], a["S0"][::2])


# ------------------------------------------------------------------------------------ convolution: runs of 16 and 32 tokens
@pytest.mark.parametrize("dtype, D, T, most", [
    (BF16, 8, 700_001, 9000),     # 16 tokens a thread: 48 KB of dynamic shared memory to the byte (W and activation as in no other test)
    (BF16, 8, 1_250_007, 20000),  # 32 tokens a thread
    (BF16, 512, 25_003, 900), (BF16, 512, 10_007, 70), (F32, 512, 15_001, 400), (F32, 40, 130_001, 3000)])
def test_packed_convolution_of_long_runs(dtype, D, T, most):
    """Sequences that begin and end anywhere in the copy groups of a run, against each sequence by itself."""
    gen = torch.Generator().manual_seed(D + T)
    lens = []
    while sum(lens) < T:
        n = int(torch.randint(0, 2 * most, (1,), generator=gen))
        lens += [min(n, T - sum(lens))] + [int(v) for v in torch.randint(0, 5, (3,), generator=gen)] * (sum(lens) + n + 12 < T)
    g = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randn(1, T, D, generator=g, device="cuda").to(dtype)
    w, s0 = torch.randn(D, 3, generator=g, device="cuda"), torch.randn(len(lens), 2, D, generator=g, device="cuda").to(dtype)
    y, end = efla.causal_conv(x, w, None, s0, cu_of(lens), activation=None)
    at = 0
    for i, n in enumerate(lens):
        y1, end1 = efla.causal_conv(x[:, at:at + n].contiguous(), w, None, s0[i:i + 1].contiguous(), activation=None)
        assert torch.equal(y[:, at:at + n], y1) and torch.equal(end[i:i + 1], end1), i
        at += n
    assert at == T and efla.device_status() == 0


# ------------------------------------------------------------------------------------ the longest rows
def need_memory(gb):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < gb * 1e9:
        pytest.skip(f"needs {gb} GB of free memory")


LONGEST = 2 ** 31 - 1 - 4096  # tokens


def test_convolution_backward_of_the_longest_row():
    """The last run ends past 2^31 - 1 places: its gradients, and its share of the sums, against its tokens by themselves."""
    need_memory(115)
    D, W, n = 8, 4, 100_000  # (all but the last n tokens are 0 and add nothing)
    gen = torch.Generator(device="cuda").manual_seed(1)
    tail = {k: torch.randn(1, n, D, generator=gen, device="cuda").to(BF16) for k in ("x", "dy")}
    long = {k: torch.zeros(1, LONGEST, D, dtype=BF16, device="cuda") for k in tail}
    for k, v in tail.items():
        long[k][:, -n:] = v
    w, dend = torch.randn(D, W, generator=gen, device="cuda"), torch.randn(1, W - 1, D, generator=gen, device="cuda").to(BF16)
    got = efla.causal_conv_bwd(long["x"], w, None, None, long["dy"], dend, activation=None)
    want = efla.causal_conv_bwd(tail["x"], w, None, None, tail["dy"], dend, activation=None)
    assert torch.equal(got["dx"][:, -n:], want["dx"]) and not bool(got["dstate0"].any())
    assert not bool(got["dx"][:, -n - 1000:-n - W + 1].any())
    ref = ssm.conv_bwd(tail["x"], w, None, None, tail["dy"], dend, silu=False)["dw"]
    size = ssm.conv_bwd(tail["x"], w, None, None, tail["dy"], dend, silu=False, size=True)["dw"]
    close(got["dw"], ref, size, n * 2.0 ** -24, "dw")  # a sum of n products
    del got, long
    torch.cuda.empty_cache()


# ------------------------------------------------------------------------------------ group norm: values far from the others or from 0
# depth: a thread's additions one after the other, those that join the threads, chunks and channels
@pytest.mark.parametrize("shape, groups, depth, whole", [
    ((20, 512), 4, 14, 16),                # a group in a warp's registers
    ((9, 4096), 2, 30, 32),                # in a team's
    ((40, 16384), 2, 38, 40),
    ((5, 64, 512), 32, 30, 32),
    ((2, 500, 8), 4, 32 * 274, 20),        # a cluster's shared memory: channels, CTAs and quotients of the mean
    ((1, 64, 64, 320), 32, 32 * 62, 20),
    ((1, 5000, 520), 5, 32 * 71, 24),      # (fp32: three kernels)
    ((1, 70001, 8), 1, 32 * 307, 20),
    ((3, 33, 2040), 1, 32 * 86, 90),       # (fp32: three kernels)
    ((2, 30000, 64), 2, 347, 4),           # three kernels
    ((1, 20000, 40), 40, 80, 4),
    ((10, 6000, 512), 512, 84, 4),         # three kernels, a warp for each of many groups
    ((4, 72000), 3, 779, 4)])
@pytest.mark.parametrize("kind", ["mean", "first"])
@pytest.mark.parametrize("dtype, silu", [(F32, True), (F32, False), (BF16, True)])
def test_group_norm_of_far_values(dtype, silu, kind, shape, groups, depth, whole):
    check_far_values(dtype, silu, kind, shape, groups, depth, whole)


@pytest.mark.parametrize("shape, groups, depth, whole", [
    ((610, 500, 8), 8, 506, 4), ((3, 100, 8), 8, 106, 4), ((610, 33, 24), 3, 39, 4), ((610, 20, 152), 4, 46, 4),  # a lane has many values
    ((700, 16, 256), 32, 22, 24), ((610, 32, 16), 4, 38, 40),                          # up to 32
    ((610, 500, 8), 1, 506, 40)])                                                      # (fp32: a team's)
@pytest.mark.parametrize("kind", ["mean", "first", "narrow"])
@pytest.mark.parametrize("dtype, silu", [(F32, True), (BF16, False)])
def test_group_norm_of_far_values_in_small_samples(dtype, silu, kind, shape, groups, depth, whole):
    """Samples that a warp takes from its memory: the mean is as good as a few roundings whatever a long sum loses."""
    check_far_values(dtype, silu, kind, shape, groups, depth, whole)


def check_far_values(dtype, silu, kind, shape, groups, depth, whole):
    x, w, b, dy = far_values(shape, groups, dtype, kind, "cuda")
    act = "silu" if silu else None
    y, stats = efla.group_norm(x, w, b, groups, activation=act, return_stats=True)
    check_stats(x, groups, stats, depth, whole)
    check_y(x, w, b, groups, silu, stats, y)
    got = efla.group_norm_bwd(x, w, b, groups, stats, dy, activation=act)
    check_gradients(x, w, b, groups, silu, stats, dy, got, depth)


@pytest.mark.parametrize("shape, groups", [((3, 0, 16), 2), ((700, 4, 0, 24), 24), ((0, 7, 16), 4)])
def test_group_norm_of_no_positions(shape, groups):
    """Statistics of nothing are NaN, as the mean of no values is, and no memory's last content."""
    stats = torch.full((shape[0], groups, 2), 7.0, device="cuda")
    x = torch.zeros(shape, device="cuda")
    y, got = efla.group_norm(x, None, None, groups, stats=stats)
    assert y.shape == x.shape and bool(got.isnan().all()) and got.data_ptr() == stats.data_ptr()
    ref = ssm.group_norm(x, None, None, groups)[1]
    assert ref.shape == got.shape and bool(ref.isnan().all())
    w = torch.ones(shape[-1], device="cuda")
    g = efla.group_norm_bwd(x, w, w, groups, stats, x)
    assert not bool(g["dw"].any()) and not bool(g["db"].any())


@pytest.mark.parametrize("call", ["conv", "scan"])
@pytest.mark.parametrize("state", [True, False])
def test_bounds_of_an_empty_batch(call, state):
    """Bounds are looked at where there are no tokens too, whether or not states are asked for."""
    for bounds, bad in (([0, 0, 0], False), ([0, 5, 0], True), ([-1, 0, 0], True)):
        cu = torch.tensor(bounds, dtype=torch.int32, device="cuda")
        if call == "conv":
            y, end = efla.causal_conv(torch.zeros(1, 0, 16, device="cuda"), torch.zeros(16, 4, device="cuda"), None, None, cu,
                                      return_state=state)
        else:
            a = scan_inputs(B=1, T=0, D=16, seqs=2)
            y, end = efla.ssm_scan(**a, cu_seqlens=cu, return_state=state)
        assert y.shape == (1, 0, 16) and (end is None) == (not state)
        assert efla.device_status() == int(bad), bounds


@pytest.mark.parametrize("bounds, exact", [
    ([0, 40, 5000, 4200, 5000], [0]), ([-3, 2500, 2600, 5001, 5000], [1]), ([10, 10, 3000, 3001, 4990], [0, 1, 2, 3]),
    ([0, 3000, 2000, 3000, 5000], []),     # more segments than 5000 tokens have: the last sequence is left out
    ([5000, 0, 5000, 0, 5000], [])])
def test_cut_sequences_around_bad_bounds(bounds, exact):
    """Malformed bounds are reported, their states left alone; a sequence is computed or left alone as a whole, unless
    another one has its tokens too; nothing else is written."""
    T, D, n = 5000, 16, len(bounds) - 1
    a = scan_inputs(B=1, T=T, D=D, seqs=n)
    cu = torch.tensor(bounds, dtype=torch.int32, device="cuda")
    need = efla.ssm_scan_workspace(1, T, D, 16, N=n)
    assert need > 0
    y, ok_y = between_sentinels(torch.full((1, T, D), 7.0, device="cuda"))
    end, ok_end = between_sentinels(torch.full((n, D, 16), 7.0, device="cuda"))
    ws, ok_ws = between_sentinels(torch.zeros(need, dtype=torch.uint8, device="cuda"))
    efla.ssm_scan(**a, cu_seqlens=cu, y=y, S_T=end, workspace=ws)
    good = [i for i in range(n) if 0 <= bounds[i] <= bounds[i + 1] <= T]
    assert efla.device_status() == int(len(good) < n)
    assert ok_y() and ok_end() and ok_ws()
    covered = torch.zeros(T, dtype=torch.int32, device="cuda")
    for i in range(n):
        if i in good:
            covered[bounds[i]:bounds[i + 1]] += 1
        else:
            assert bool((end[i] == 7).all())
    assert bool((y[0, covered == 0] == 7).all())
    for i in good:
        lo, hi = bounds[i:i + 2]
        if bool((covered[lo:hi] > 1).any()):
            continue
        if i not in exact and bool((end[i] == 7).all()):
            assert bool((y[0, lo:hi] == 7).all()), i
            continue
        one = {k: v[:, lo:hi].contiguous() if k in ("x", "dt", "B", "C", "z") else v for k, v in a.items()}
        one["S0"] = a["S0"][i:i + 1].contiguous()
        ref, ref_S = ssm.scan(**one)
        size, size_S = ssm.scan(**one, size=True)
        close(y[:, lo:hi], ref, size, scan_share(hi - lo), f"y {i}")
        close(end[i:i + 1], ref_S, size_S, scan_share(hi - lo), f"S {i}")
