"""The bound that the weight gradients are held to (tree_plain.check_weight_grad)
sees a lost or doubled group of rows: mistakes planted in the 64-bit form."""
import numpy as np
import pytest
import torch

from tests import tree_plain as tp

EPS = 1e-5


@pytest.mark.parametrize("T,H,other,D,rot", [(6001, 16, 1, 64, 48), (4003, 8, 2, 128, 112)])
def test_planted_mistakes_are_seen(T, H, other, D, rot):
    g = torch.Generator().manual_seed(T)
    x, gr = (torch.randn(T, H, D, generator=g).bfloat16() for _ in range(2))
    w = (1 + 0.3 * torch.randn(D, generator=g)).bfloat16()
    f = (10000.0 ** (-2 * torch.arange(rot // 2, dtype=torch.float64) / rot)).float()
    ang = tp.angles(torch.randint(0, 5000, (T,), generator=g).numpy(), f)
    adds = tp.lane_additions(T, H, other, D, 152)
    args = (x, w, gr, ang, EPS, False, adds)
    part = lambda a, b: tp.norm_rope_grad(x[a:b], w, gr[a:b], ang[a:b], EPS, False)[1]  # noqa: E731
    right = part(0, T)
    tp.check_weight_grad(torch.from_numpy(right.astype(np.float32)), *args)
    one_row = tp.norm_rope_grad(x[5:6, :1], w, gr[5:6, :1], ang[5:6], EPS, False)[1]
    for mistake in (-part(T - 16, T), part(T - 16, T), -part(T - 1, T), part(100, 101), -one_row):
        with pytest.raises(AssertionError, match="weight gradient off"):
            tp.check_weight_grad(torch.from_numpy((right + mistake).astype(np.float32)), *args)
