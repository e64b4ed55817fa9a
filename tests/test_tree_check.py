"""The bounds that the tree's attention is held to (tree_plain.check_tree) see a
wrong mask, length or row: mistakes planted in the 64-bit form."""
import random

import numpy as np
import pytest
import torch

from tests import tree_plain as tp


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_planted_mistakes_are_seen(dtype):
    B, N, Hq, Hkv, D, page, lens = 2, 9, 4, 2, 64, 32, [75, 60]
    g = torch.Generator().manual_seed(1)
    kp, vp = (torch.randn(7, page, Hkv, D, generator=g).to(dtype) for _ in range(2))
    q = torch.randn(B, N, Hq, D, generator=g).to(dtype)
    table = np.array([[2, 0, 5], [1, 6, 3]])
    parents = tp.random_parents(B, N, random.Random(2))
    scale = D ** -0.5
    right = (kp, vp, table, lens, parents)

    def check(kp, vp, table, lens, parents):
        O, lse, _, _ = tp.decode_tree(q, kp, vp, table, lens, parents, scale)
        tp.check_tree(torch.from_numpy(O).to(dtype), torch.from_numpy(lse).float(), q, *right, scale)

    check(*right)
    cousin = [list(p) for p in parents]
    cousin[0][8] = 0 if cousin[0][8] else 1  # another way to the root
    extra = [list(p) for p in parents]
    extra[1][5] = 4 if extra[1][5] != 4 else 3  # one more, or another, ancestor
    stale = kp.clone()
    t = lens[0] - N + 3  # node 3's key left as another slot's
    stale[table[0][t // page], t % page] = kp[table[0][0], 0]
    swapped = table.copy()
    swapped[1] = swapped[1][[1, 0, 2]]
    for mistake in ((kp, vp, table, lens, cousin), (kp, vp, table, lens, extra),
                    (kp, vp, table, [74, 60], parents), (kp, vp, table, [75, 59], parents),
                    (stale, vp, table, lens, parents), (kp, vp, swapped, lens, parents)):
        with pytest.raises(AssertionError, match="off by"):
            check(*mistake)
