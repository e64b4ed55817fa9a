"""Attention with shared prefixes (fa_decode_shared_fwd) where the plan has more groups and
sequences than a block has threads: streamed and tiled sequences of both head sizes against
the plain form, and long prefixes cut into strips against the paged decode."""
import random

import pytest
import torch

from tests.test_decode_shared_gpu import check, inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hq,Hkv,D,Sq,dtype", [
    (12, 1, 128, 1, torch.bfloat16),   # 12 rows: streamed
    (20, 1, 128, 1, torch.float16),    # 20 rows: a tile of its own
    (6, 2, 64, 6, torch.bfloat16),     # 18 rows
    (70, 1, 128, 2, torch.bfloat16),   # 140 rows: two row tiles
])
def test_many_owners(fa, Hq, Hkv, D, Sq, dtype):
    rng = random.Random(Hq)
    starts, lens, prefix = [0], [], []
    for i in range(220):
        n = rng.choice([1, 1, 2, 3, 4 if i % 20 else 16])
        P = rng.choice([0, 20, 33, 64, 129])
        starts.append(starts[-1] + n)
        prefix.append(P)
        lens += [P + rng.choice([0, Sq, Sq + 1, 40]) for _ in range(n)]
    lens += [rng.choice([0, 1, 50]) for _ in range(3)]   # in no group
    assert len(prefix) + len(lens) > 384
    check(fa, inputs(Hq, Hkv, D, 32, starts, prefix, lens, Sq, dtype, seed=Hq), D ** -0.5)


@pytest.mark.parametrize("Hkv,G,D,Sq,P,members,others", [
    (8, 16, 128, 2, 13001, 20, 400),  # 640 rows behind 102 tiles: strips; 32 rows of each other
    (8, 8, 64, 1, 25000, 40, 400),    # 320 rows behind 196 tiles; 8 rows of each other: streamed
])
def test_strips_among_many_owners(fa, Hkv, G, D, Sq, P, members, others):
    """|V| <= 1, so each O is off by P's rounding, 2^-8, and its own; log-sum-exps by the scores'
    fp32 sums, |q| |k| scale (D + 4) 2^-24, and 2^-18."""
    rng, page, dev = random.Random(P), 64, "cuda"
    g = torch.Generator(device=dev).manual_seed(P)
    before = others // 2
    lens = ([rng.randint(1, 300) for _ in range(before)] + [P + rng.randint(Sq, 300) for _ in range(members)]
            + [rng.randint(1, 300) for _ in range(others - before)])
    B, whole, used = len(lens), P // page, P // page
    rows = []
    for b, L in enumerate(lens):
        shared = list(range(whole)) if before <= b < before + members else []
        more = -(-L // page) - len(shared)
        rows.append(shared + list(range(used, used + more)))
        used += more
    width = max(len(r) for r in rows)
    kp = torch.randn(used, page, Hkv, D, generator=g, device=dev).bfloat16()
    vp = (2 * torch.rand(used, page, Hkv, D, generator=g, device=dev) - 1).bfloat16()
    r, first = P % page, rows[before]
    for row in rows[before + 1:before + members]:
        kp[row[whole], :r] = kp[first[whole], :r]
        vp[row[whole], :r] = vp[first[whole], :r]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    table, ln = i32([x + [0] * (width - len(x)) for x in rows]), i32(lens)
    q = torch.randn(B, Sq, Hkv * G, D, generator=g, device=dev).bfloat16()
    scale = D ** -0.5
    a, la = fa.decode_paged(q, kp, vp, table, ln, scale, lse=True)
    args = (q, kp, vp, table, ln, i32([before, before + members]), i32([P]), scale)
    b, lb = fa.decode_shared(*args, lse=True)
    again = fa.decode_shared(*args)
    torch.cuda.synchronize()
    assert fa.fa_device_error()[0] == fa.FA_OK
    assert torch.equal(b, again)
    assert ((a.double() - b.double()).abs() <= 2 * 2.0 ** -8 * (1.0 + a.double().abs()) * 1.02).all()
    dead = torch.isneginf(la)
    assert torch.equal(dead, torch.isneginf(lb))
    qk = float(q.float().norm(dim=-1).max() * kp.float().norm(dim=-1).max())
    assert ((la - lb)[~dead].abs() <= 2 * ((D + 4) * 2.0 ** -24 * scale * qk + 2.0 ** -18)).all()
