"""A paged cache's bookkeeping (fa_update_pages) and row writes (fa_write_pages):
whole numbers and copies, which have to be equal to the plain forms'."""
import random

import pytest
import torch

from tests import serving_plain as sp

pytestmark = pytest.mark.gpu


def inputs(B, page, width, seed, kinds=("grow", "new", "end", "shrink", "same"), spare=10, most=None,
           shared=False):
    rng = random.Random(seed)
    cap = width * page
    old, new, sh = [], [], []
    for _ in range(B):
        o = rng.choice([0, 1, page - 1, page, page + 1, rng.randint(0, cap), cap])
        o = min(o, cap)
        k = rng.choice(kinds)
        if k == "new":
            o, n = 0, rng.randint(0, min(cap, most or cap))
        elif k == "end":
            n = 0
        elif k == "shrink":
            n = rng.randint(0, o)
        elif k == "grow":
            n = min(cap, o + rng.choice([1, 1, 2, page, rng.randint(0, most or cap)]))
        else:
            n = o
        old.append(o)
        new.append(n)
        sh.append(rng.choice([0, 0, 1, 2, width]) if shared else 0)
    held = [max(-(-o // page), s) for o, s in zip(old, sh)]
    total = sum(held) + spare
    ids = list(range(total))
    rng.shuffle(ids)
    table = [[-7] * width for _ in range(B)]
    at = 0
    for b, n in enumerate(held):
        table[b][:n] = ids[at:at + n]
        at += n
    stack = ids[at:] + [-5] * at
    return table, old, new, stack, total - at, (sh if shared else None)


def run(fa, table, old, new, stack, count, page, max_new, shared=None, in_place=False, status=None):
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    t, st, o, c = i32(table).reshape(len(old), len(table[0]) if table else 1), i32(stack), i32(old), i32([count])
    lens, left, cu, slots, pos = fa.update_pages(
        t, o, i32(new), st, c, page, max_new, shared_pages=None if shared is None else i32(shared),
        lens_out=o if in_place else None, free_count_out=c if in_place else None)
    torch.cuda.synchronize()
    got, detail = fa.fa_device_error()
    want = sp.update_pages(table, old, new, stack, count, page, max_new, shared)
    assert got == (fa.FA_ERR_BOUNDS if want[7] else fa.FA_OK), hex(detail)
    if in_place:
        assert lens.data_ptr() == o.data_ptr() and left.data_ptr() == c.data_ptr()
    else:
        assert o.tolist() == list(old) and c.tolist() == [count]
    assert lens.tolist() == want[2] and left.tolist() == [want[3]]
    assert cu.tolist() == want[4]
    assert t.tolist() == want[0]
    assert st.tolist() == want[1]
    assert slots.tolist() == want[5] and pos.tolist() == want[6]
    return want


@pytest.mark.parametrize("B,page,width,spare", [
    (1, 32, 1, 1), (1, 64, 9, 30), (5, 96, 4, 60), (64, 64, 20, 2000), (300, 32, 7, 4000),
    (511, 32, 3, 3000), (512, 64, 3, 3000), (513, 32, 5, 5000), (1500, 32, 2, 9000), (4096, 32, 2, 20000),
])
@pytest.mark.parametrize("in_place", [False, True])
def test_update(fa, B, page, width, spare, in_place):
    table, old, new, stack, count, _ = inputs(B, page, width, seed=B + page, spare=spare)
    tokens = sum(max(0, n - o) for o, n in zip(old, new))
    want = run(fa, table, old, new, stack, count, page, tokens + 5, in_place=in_place)
    assert want[2] == new  # (there was room)


@pytest.mark.parametrize("seed", range(8))
def test_not_enough_pages_or_slots(fa, seed):
    """Sequences that find no room keep their lengths, and later ones that need no page
    go on; what is given back in the same call is taken again."""
    table, old, new, stack, count, sh = inputs(70, 32, 6, seed=seed, spare=seed * 9, shared=seed % 2 == 1)
    tokens = sum(max(0, n - o) for o, n in zip(old, new))
    run(fa, table, old, new, stack, count, 32, max(0, tokens - seed % 3 * 200), sh, in_place=True)


def test_long_prompts_over_the_whole_cluster(fa):
    table, old, new, stack, count, _ = inputs(9, 128, 300, seed=2, kinds=("new", "grow", "end"), spare=3000)
    tokens = sum(max(0, n - o) for o, n in zip(old, new))
    run(fa, table, old, new, stack, count, 128, tokens + 3)


def test_shared_pages_are_not_taken_given_or_written(fa):
    page = 32
    table = [[3, 4, -7, -7], [3, 4, 9, -7], [3, 4, 5, 6]]
    want = run(fa, table, [64, 70, 128], [100, 0, 64], [20, 21, 22, -1, -1, -1, -1], 3, page, 40,
               shared=[2, 2, 2])
    assert want[0][0][:4] == [3, 4, 6, 5]  # what the third gave back last, then what before
    # A sequence that starts inside its shared pages gets no slots there.
    want = run(fa, [[3, 4, -7]], [40], [70], [8], 1, page, 40, shared=[2])
    assert want[5][:24] == [-1] * 24 and want[5][24:30] == [8 * 32 + i for i in range(6)]


def test_empty(fa):
    run(fa, [], [], [], [1, 2], 2, 32, 5)
    run(fa, [[-7]], [0], [0], [1, 2], 2, 32, 0)
    run(fa, [[-7]], [0], [3], [], 0, 32, 9)  # no free page at all


@pytest.mark.parametrize("old,new,shared,count", [
    ([5, -1, 9], [6, 4, 10], None, 4), ([5, 40, 9], [6, 97, 10], None, 4), ([97, 1, 1], [6, 2, 2], None, 4),
    ([5, 4, 9], [6, -2, 10], None, 4), ([5, 4, 9], [6, 5, 10], [0, 4, 0], 4),
    ([5, 4, 9], [6, 5, 10], [0, -1, 0], 4), ([5, 4, 9], [6, 5, 10], None, 7), ([5, 4, 9], [6, 5, 10], None, -1),
    ([5, 96, 96], [6, 0, 0], None, 4),  # more comes back than the stack holds
])
def test_lengths_and_counts_that_cannot_be(fa, old, new, shared, count):
    table = [[0, 1, 2], [3, 4, 5], [6, 7, 8]]
    want = run(fa, table, old, new, [10, 11, 12, 13, -1, -1], count, 32, 20, shared)
    assert want[7]
    assert fa.fa_device_error()[0] == fa.FA_OK


def test_page_ids_without_a_slot(fa):
    want = run(fa, [[2 ** 26, -3]], [30], [36], [11], 1, 32, 9)
    assert want[7] and want[5][:6] == [-1, -1, 352, 353, 354, 355]


# ---------------------------------------------------------------- rows
@pytest.mark.parametrize("T,Hkv,D,page,dtype", [
    (1, 1, 64, 32, torch.bfloat16), (3, 2, 128, 96, torch.float16), (257, 5, 64, 64, torch.bfloat16),
    (1000, 8, 128, 32, torch.float16), (33, 16, 128, 256, torch.bfloat16),
])
@pytest.mark.parametrize("packed", [False, True])
def test_write(fa, T, Hkv, D, page, dtype, packed):
    g = torch.Generator().manual_seed(T)
    pages = -(-T // page) + 2
    kp, vp = (torch.randn(pages, page, Hkv, D, generator=g).to(dtype) for _ in range(2))
    if packed:
        x = torch.randn(T, 3 * Hkv + 1, D, generator=g).to(dtype)
        k, v = x[:, 1:Hkv + 1], x[:, 2 * Hkv + 1:]
    else:
        k, v = (torch.randn(T, Hkv, D, generator=g).to(dtype) for _ in range(2))
    slots = torch.randperm(pages * page, generator=g)[:T].int()
    slots[::7] = -1
    kd, vd, kpd, vpd = (t.cuda() for t in (k, v, kp, vp))
    if packed:
        xd = x.cuda()
        kd, vd = xd[:, 1:Hkv + 1], xd[:, 2 * Hkv + 1:]
    fa.write_pages(kd, vd, kpd, vpd, slots.cuda())
    torch.cuda.synchronize()
    assert fa.fa_device_error()[0] == fa.FA_OK
    for t, s in enumerate(slots.tolist()):
        if s >= 0:
            kp[s // page, s % page], vp[s // page, s % page] = k[t], v[t]
    assert torch.equal(kpd.cpu().view(torch.int16), kp.view(torch.int16))
    assert torch.equal(vpd.cpu().view(torch.int16), vp.view(torch.int16))


def test_slots_past_the_cache_are_skipped_and_reported(fa):
    kp = torch.zeros(2, 32, 1, 64, dtype=torch.bfloat16, device="cuda")
    vp, k = kp.clone(), torch.ones(4, 1, 64, dtype=torch.bfloat16, device="cuda")
    slots = torch.tensor([0, 64, -9, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    fa.write_pages(k, k, kp, vp, slots)
    assert fa.fa_device_error()[0] == fa.FA_ERR_BOUNDS
    assert kp[0, 0].eq(1).all() and kp.sum() == 64 and torch.equal(kp, vp)


def test_write_past_2_to_31_elements(fa):
    """Slots whose elements lie past 2^31 in the cache (9 GB of pages)."""
    Hkv, D, page = 16, 128, 256
    pages = 2 ** 31 // (page * Hkv * D) + 8
    kp = torch.zeros(pages, page, Hkv, D, dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    k = torch.randn(5, Hkv, D, device="cuda").bfloat16()
    at = [pages * page - 1, pages * page - 300, 2 ** 31 // (Hkv * D), 2 ** 31 // (Hkv * D) - 1, 0]
    fa.write_pages(k, -k, kp, vp, torch.tensor(at, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    flat, vflat = kp.view(-1, Hkv, D), vp.view(-1, Hkv, D)
    for t, s in enumerate(at):
        assert torch.equal(flat[s], k[t]) and torch.equal(vflat[s], -k[t])
    assert int((flat != 0).any(-1).any(-1).sum()) == 5
    assert fa.fa_device_error()[0] == fa.FA_OK
