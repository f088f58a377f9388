"""Bounds of a group norm's results that hold however far a group's mean is from 0 or one value from the others.

`depth`: the additions that a sum over a group's values goes through one after the other (times 32 where squares are not taken
from the mean but from a value up to five and a half deviations from it: 1 + 5.6^2).  `whole`: the roundings of sums of values themselves, not of
differences, on the way to the mean.  The forward's statistics are held
to x's own in 64 bits, y and the gradients to the formulas in 64 bits with the forward's own statistics, so that what a mean
rounded to fp32 does to n (2^-24 |mean| / sigma) is allowed once, in the mean, and nowhere else.
"""
import torch

from oracle import ssm

U = 2.0 ** -24


def over(got, ref, tol):
    """By how much got is further from ref than tol (and, for bf16, half a step) at worst; NaN counts as infinitely far."""
    step = 2.0 ** -8 if got.dtype == torch.bfloat16 else 0.0
    d = (got.double() - ref).abs() - step * ref.abs() - tol
    return float(torch.nan_to_num(d, nan=float("inf")).max())


def check_stats(x, groups, stats, depth, whole, eps=1e-5):
    xg = x.double().reshape(x.shape[0], -1, groups, x.shape[-1] // groups)
    mean = xg.mean((1, 3), keepdim=True)
    away = (xg - mean).abs().mean((1, 3))
    var = ((xg - mean) ** 2).mean((1, 3))
    mean = mean[:, 0, :, 0]
    # (a first mean is off by less than `away`, so the differences from it are twice that at most)
    tol = whole * U * xg.abs().mean((1, 3)) + 2 * (depth + 4) * U * away + 1e-30
    assert over(stats[..., 0], mean, tol) <= 0, ("mean", over(stats[..., 0], mean, tol))
    # a sum of positive terms: depth roundings, six of each term and of the quotient, four of the inverse root; measured from
    # a mean that is off by tol it is tol^2 larger
    r = 1 / torch.sqrt(var + eps)
    share = (0.5 * depth + 10) * U + 0.5 * (tol * r) ** 2
    assert over(stats[..., 1], r, share * r) <= 0, ("r", float(((stats[..., 1] - r) / r).abs().max()), float(share.max()))


def check_y(x, w, b, groups, silu, stats, y):
    """n, w n and + b: five roundings of the parts' size; silu: a sigmoid of 2 + 1.2 |s| ulp (7e-7 for |s| < 8), slope 1.1."""
    n = ssm.group_norm(x, None, None, groups, stats=stats)[0].abs()
    size = (n if w is None else n * w.abs()) + (0 if b is None else b.abs())
    ref = ssm.group_norm(x, w, b, groups, silu=silu, stats=stats)[0]
    tol = 1.1 * (5 * U + (7e-7 if silu else 0)) * size + 1e-30
    assert over(y, ref, tol) <= 0, ("y", over(y, ref, tol))


def check_gradients(x, w, b, groups, silu, stats, dy, got, depth):
    """Sums over a group of depth `depth`, over all positions of as many additions as there are; the elementwise parts 20
    roundings, the activation's slope four sigmoids."""
    ref, size = ssm.group_norm_bwd(x, w, b, groups, dy, silu=silu, stats=stats)
    many = x.numel() // x.shape[-1]
    for name, v in ref.items():
        if v is None:
            assert got[name] is None
            continue
        share = ((depth if name == "dx" else many) + 20) * U + (2.8e-6 if silu else 0)
        assert over(got[name], v, share * size[name] + 1e-30) <= 0, (name, over(got[name], v, share * size[name]))


def far_values(shape, groups, dtype, kind, device, seed=0):
    """Groups whose values are far from 0 ("mean"), nearly equal as well ("narrow"), or whose first position is far from
    the others ("first")."""
    gen = torch.Generator(device=device).manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=gen, device=device)  # noqa: E731
    C = shape[-1]
    x = rand(*shape) * (0.5 + torch.rand(C, generator=gen, device=device)) + 0.5 * rand(C)
    if kind == "mean":
        x = x + 300
    elif kind == "narrow":
        x = 30000.3 + 0.05 * x
    elif len(shape) == 2:
        x[:, ::C // groups] = 1000
    else:
        x.view(shape[0], -1, C)[:, 0] = 1000
    w, b = rand(C), rand(C)
    return x.to(dtype), w, b, rand(*shape).to(dtype)
