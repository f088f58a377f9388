"""The bounds of norm_bounds.py hold for a careful fp32 norm and reject what they are there to reject."""
import pytest
import torch

from norm_bounds import check_gradients, check_stats, check_y, far_values
from oracle import ssm

SHAPE, GROUPS = (2, 300, 64), 2


def stats_of(x, naive):
    """Statistics in fp32: the mean and the deviations from it, or the mean of squares less the square of the mean."""
    xg = x.float().reshape(x.shape[0], -1, GROUPS, x.shape[-1] // GROUPS).transpose(1, 2).flatten(2)
    near = xg[..., :1]
    mean = (near + (xg - near).mean(-1, keepdim=True))
    var = (xg * xg).mean(-1) - mean[..., 0] ** 2 if naive else ((xg - mean) ** 2).mean(-1)
    return torch.stack([mean[..., 0], 1 / torch.sqrt(var + 1e-5)], -1)


@pytest.mark.parametrize("kind", ["mean", "first"])
def test_bounds_of_the_statistics(kind):
    x, w, b, dy = far_values(SHAPE, GROUPS, torch.float32, kind, "cpu")
    check_stats(x, GROUPS, stats_of(x, False), 100, 4)
    if kind == "mean":
        with pytest.raises(AssertionError, match="'r'"):
            check_stats(x, GROUPS, stats_of(x, True), 100, 4)
    off = stats_of(x, False)
    off[..., 0] *= 1 + 2.0 ** -20  # (16 roundings of the mean)
    if kind == "mean":
        with pytest.raises(AssertionError, match="mean"):
            check_stats(x, GROUPS, off, 100, 4)


@pytest.mark.parametrize("kind", ["mean", "first"])
def test_bounds_of_the_results(kind):
    x, w, b, dy = far_values(SHAPE, GROUPS, torch.float32, kind, "cpu")
    stats = stats_of(x, False)
    y, _ = ssm.group_norm(x, w, b, GROUPS, silu=True, stats=stats)
    got, _ = ssm.group_norm_bwd(x, w, b, GROUPS, dy, silu=True, stats=stats)
    got = {k: v.float() for k, v in got.items()}
    check_y(x, w, b, GROUPS, True, stats, y.float())
    check_gradients(x, w, b, GROUPS, True, stats, dy, got, 100)
    with pytest.raises(AssertionError, match="'y'"):
        check_y(x, w, b, GROUPS, True, stats, y.float() * (1 + 1e-5))
    for name in got:
        with pytest.raises(AssertionError, match=name):
            check_gradients(x, w, b, GROUPS, True, stats, dy, got | {name: torch.zeros_like(got[name])}, 100)
    half = ssm.group_norm_bwd(x, w, b, GROUPS, dy, silu=True, stats=stats * torch.tensor([1.0, 1.0 + 1e-4]))[0]
    with pytest.raises(AssertionError, match="dx"):
        check_gradients(x, w, b, GROUPS, True, stats, dy, {k: v.float() for k, v in half.items()}, 100)
