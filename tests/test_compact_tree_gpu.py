"""Compaction of accepted paths in a paged cache (fa_compact_tree): copies, so
every bit of the pools and every length has to be equal."""
import random

import pytest
import torch

from tests import tree_plain as tp

pytestmark = pytest.mark.gpu


def inputs(B, N, layers, Hkv, D, page, lens, dtype, seed, keep=None):
    rng = random.Random(seed)
    g = torch.Generator().manual_seed(seed)
    max_pages = max(1, -(-max(lens + [1]) // page))
    num_pages = B * max_pages + 2
    shape = (layers, num_pages, page, Hkv, D)
    k, v = torch.randn(shape, generator=g).to(dtype), torch.randn(shape, generator=g).to(dtype)
    table = torch.randperm(num_pages, generator=g)[:B * max_pages].reshape(B, max_pages).int()
    path, count = [], []
    for b in range(B):
        n = rng.randint(0, N) if keep is None else keep
        path.append(sorted(rng.sample(range(N), n)) + [-1] * (N - n))
        count.append(n)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    return k, v, table, i32(lens), i32(path), i32(count)


def check(fa, t, status=None, in_place=False, squeeze=False):
    k, v, table, lens, path, count = t
    N = path.shape[1]
    kd, vd, ld = k.cuda(), v.cuda(), lens.cuda()
    got = fa.compact_tree(kd[0] if squeeze else kd, vd[0] if squeeze else vd, table.cuda(), ld,
                          path.cuda(), count.cuda(), seqlens_out=ld if in_place else None)
    torch.cuda.synchronize()
    st, detail = fa.fa_device_error()
    assert st == (fa.FA_OK if status is None else status), hex(detail)
    k, v = k.clone(), v.clone()
    for pool, dev in ((k, kd), (v, vd)):
        want = tp.compact(pool, table.numpy(), lens.tolist(), path.tolist(), count.tolist(), N)
        assert torch.equal(dev.cpu().view(torch.int16), pool.view(torch.int16))
    assert got.tolist() == want
    if in_place:
        assert ld.tolist() == want


@pytest.mark.parametrize("B,N,layers,Hkv,D,page,lens,dtype", [
    (1, 1, 1, 1, 64, 32, [1], torch.bfloat16),
    (1, 8, 1, 2, 128, 64, [2733], torch.bfloat16),
    (4, 64, 3, 5, 64, 32, [64, 65, 200, 95], torch.float16),    # trees over three pages
    (3, 16, 2, 8, 128, 96, [16, 0, 101], torch.bfloat16),       # padding among them
    (40, 7, 1, 1, 64, 32, [7 + 3 * i for i in range(40)], torch.bfloat16),
])
@pytest.mark.parametrize("in_place", [False, True])
def test_compact(fa, B, N, layers, Hkv, D, page, lens, dtype, in_place):
    check(fa, inputs(B, N, layers, Hkv, D, page, lens, dtype, seed=N + B), in_place=in_place)


def test_one_layer_without_the_axis(fa):
    check(fa, inputs(2, 12, 1, 2, 64, 64, [70, 130], torch.float16, seed=1), squeeze=True)


def test_whole_tree_and_nothing(fa):
    check(fa, inputs(2, 20, 1, 2, 64, 32, [70, 130], torch.bfloat16, seed=2, keep=20))
    check(fa, inputs(2, 20, 1, 2, 64, 32, [70, 130], torch.bfloat16, seed=3, keep=0))


@pytest.mark.parametrize("in_place", [False, True])
def test_bad_paths_lengths_and_pages_leave_the_sequence(fa, in_place):
    t = list(inputs(7, 6, 2, 2, 64, 32, [50, 60, 70, 80, 90, 64, 31], torch.bfloat16, seed=4, keep=3))
    k, v, table, lens, path, count = t
    path[0] = torch.tensor([0, 4, 2, -1, -1, -1])   # does not rise
    path[1] = torch.tensor([0, 6, 7, -1, -1, -1])   # no such node
    count[2] = 7
    count[3] = -1
    path[4] = torch.tensor([1, 3, 5, -1, -1, -1])
    table[4, 2] = 10 ** 6                           # a page that does not exist
    lens[5] = 97                                    # past the page table
    check(fa, tuple(t), status=fa.FA_ERR_BOUNDS, in_place=in_place)
    assert fa.fa_device_error()[0] == fa.FA_OK
