"""Attention of a batch whose sequences share prefixes (fa_decode_shared_fwd) against a
plain 64-bit form of every sequence by itself: rows around one and two row tiles,
prefixes and lengths around the tile and page edges, several groups, sequences in none,
alone, empty or not past their prefix, NaN wherever nothing may be read, bad inputs."""
import math
import random

import pytest
import torch

from tests import serving_plain as sp

pytestmark = pytest.mark.gpu


def inputs(Hq, Hkv, D, page, starts, prefix, lens, Sq, dtype, seed, width=None):
    """Shuffled pages; slots that hold no token are NaN, and so are the copies of a
    prefix's end that sequences past it have in pages of their own."""
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    width = width or max(1, -(-max(max(lens), 1) // page))
    pages = B * width + 3
    ids = torch.randperm(pages, generator=g).tolist()
    kp = torch.full((pages, page, Hkv, D), float("nan"), dtype=dtype)
    vp = kp.clone()
    table = torch.full((B, width), 10 ** 6, dtype=torch.int32)

    def fill(b, t, k, v):
        kp[int(table[b, t // page]), t % page] = k
        vp[int(table[b, t // page]), t % page] = v

    own = 0
    for b, L in enumerate(lens):
        gi = [i for i in range(len(prefix)) if starts[i] <= b < starts[i + 1]]
        P = prefix[gi[0]] if gi else 0
        over = [x for x in range(starts[gi[0]], starts[gi[0] + 1]) if lens[x] - Sq + 1 >= P] if gi else []
        past = gi and starts[gi[0] + 1] - starts[gi[0]] > 1 and b in over
        first = over[0] if past else b
        common = P // page if past and b != first else 0
        for j in range(-(-max(L, 0) // page)):
            if j < common:
                table[b, j] = table[first, j]
            else:
                table[b, j] = ids[own]
                own += 1
        gp = torch.Generator().manual_seed(seed * 1000 + (gi[0] if gi else 500 + b))
        pk = torch.randn(max(P, 1), Hkv, D, generator=gp).to(dtype)
        pv = torch.randn(max(P, 1), Hkv, D, generator=gp).to(dtype)
        for t in range(min(max(L, 0), width * page)):
            if t < P:
                if not (past and b != first and t // page >= common):
                    fill(b, t, pk[t], pv[t])
            else:
                fill(b, t, torch.randn(Hkv, D, generator=g).to(dtype), torch.randn(Hkv, D, generator=g).to(dtype))
    q = torch.randn(B, Sq, Hq, D, generator=g).to(dtype)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    return q, kp, vp, table, i32(lens), i32(starts), i32(prefix)


def whole(t):
    """The same cache with every sequence's tokens in pages of its own, for the plain form."""
    q, kp, vp, table, lens, starts, prefix = t
    B, width, page = table.shape[0], table.shape[1], kp.shape[1]
    k2 = torch.full((B * width,) + kp.shape[1:], float("nan"), dtype=kp.dtype)
    v2, t2 = k2.clone(), torch.arange(B * width, dtype=torch.int32).reshape(B, width)
    for b in range(B):
        gi = [i for i in range(len(prefix)) if starts[i] <= b < starts[i + 1]]
        P = int(prefix[gi[0]]) if gi else 0
        over = [x for x in range(starts[gi[0]], starts[gi[0] + 1])
                if int(lens[x]) - q.shape[1] + 1 >= P] if gi else []
        past = gi and starts[gi[0] + 1] - starts[gi[0]] > 1 and b in over
        for tok in range(min(max(int(lens[b]), 0), width * page)):
            r = over[0] if past and tok < P else b
            src = int(table[r, tok // page])
            k2[b * width + tok // page, tok % page] = kp[src, tok % page]
            v2[b * width + tok // page, tok % page] = vp[src, tok % page]
    return q, k2, v2, t2, lens


def run(fa, t, scale, status=None):
    out, lse = fa.decode_shared(*(x.cuda() for x in t), scale, lse=True)
    torch.cuda.synchronize()
    st, detail = fa.fa_device_error()
    assert st == (fa.FA_OK if status is None else status), hex(detail)
    return out, lse


def check(fa, t, scale, status=None):
    out, lse = run(fa, t, scale, status)
    q, k2, v2, t2, lens = whole(t)
    sp.check_decode(out, lse, q, k2, v2, t2.numpy(), lens.tolist(), scale)
    return out, lse


@pytest.mark.parametrize("Hq,Hkv,D,page,starts,prefix,lens,Sq,dtype", [
    (2, 1, 64, 32, [0, 2], [1], [1, 2], 1, torch.bfloat16),                  # a prefix of one token
    (4, 2, 128, 64, [0, 3], [127], [127, 128, 300], 1, torch.float16),       # nothing of its own
    (8, 1, 64, 32, [0, 4], [128], [129, 140, 128, 500], 1, torch.bfloat16),  # prefix ends with a tile
    (8, 2, 128, 96, [0, 5], [400], [401, 402, 530, 800, 410], 1, torch.float16),
    (16, 1, 128, 64, [0, 8], [260], [261 + 37 * i for i in range(8)], 1, torch.bfloat16),   # 128 rows
    (43, 1, 64, 32, [0, 3], [515], [516, 600, 555], 1, torch.bfloat16),      # 129 rows: a second tile of one
    (16, 1, 128, 32, [0, 16], [700], [701 + 9 * i for i in range(16)], 1, torch.float16),   # 256 rows
    (16, 1, 64, 64, [0, 17], [390], [391 + 5 * i for i in range(17)], 1, torch.bfloat16),   # 272: one more tile
    (24, 1, 128, 64, [0, 16], [333], [340 + 5 * i for i in range(16)], 1, torch.bfloat16),  # 384 rows
    (14, 2, 64, 256, [0, 6], [257], [300, 262, 700, 264, 265, 266], 4, torch.float16),      # new tokens, odd group
    (64, 1, 128, 64, [0, 3], [200], [203, 260, 331], 3, torch.bfloat16),     # 192 rows of one sequence
    (64, 1, 64, 32, [0, 2], [150], [158, 400], 8, torch.float16),            # 512 rows of one sequence
    (6, 6, 128, 32, [0, 4], [90], [95, 96, 97, 200], 2, torch.float16),      # MHA
])
def test_one_group(fa, Hq, Hkv, D, page, starts, prefix, lens, Sq, dtype):
    check(fa, inputs(Hq, Hkv, D, page, starts, prefix, lens, Sq, dtype, seed=Hq + D), 1 / math.sqrt(D))


@pytest.mark.parametrize("groups", [0, 1, 4])
def test_sequences_in_no_group(fa, groups):
    """Before the first start, behind the last, and with no groups at all."""
    starts = [2, 4, 4, 7, 9][:groups + 1] if groups else [5]
    prefix = [130, 70, 257, 96][:groups]
    lens = [300, 1, 140, 131, 280, 258, 259, 96, 200, 0, 77]
    check(fa, inputs(8, 2, 64, 32, starts, prefix, lens, 1, torch.bfloat16, seed=groups), 0.125)


def test_members_alone_short_empty_and_not_past_the_prefix(fa):
    starts, prefix = [0, 1, 5, 9, 12], [200, 300, 128, 0]
    lens = [260, 301, 299, 300, 302, 0, 5, 128, 400, 0, 0, 0]
    check(fa, inputs(4, 2, 128, 32, starts, prefix, lens, 1, torch.float16, seed=3), 0.09)
    lens = [260, 305, 301, 303, 302, 3, 5, 131, 400, 2, 4, 1]  # three new tokens
    check(fa, inputs(4, 2, 64, 32, starts, prefix, lens, 3, torch.bfloat16, seed=4), 0.125)


def test_all_empty(fa):
    t = inputs(4, 2, 64, 32, [0, 3], [0], [0, 0, 0], 2, torch.bfloat16, seed=5, width=2)
    out, lse = check(fa, t, 0.125)
    assert not out.any() and torch.isneginf(lse).all()


@pytest.mark.parametrize("seed", range(8))
def test_shares_that_end_anywhere(fa, seed):
    """Groups and sequences of all sizes: ranges of the list that begin and end in the
    middle of strips, between them, and in none."""
    rng = random.Random(seed)
    Hkv, Sq = rng.choice([1, 2, 3]), rng.choice([1, 1, 2, 5])
    Hq = Hkv * rng.choice([1, 4, 7, 16])
    n = rng.choice([1, 2, 5, 9])
    sizes = [rng.choice([1, 2, 3, rng.randint(1, 12)]) for _ in range(n)]
    starts = [0]
    for s in sizes:
        starts.append(starts[-1] + s)
    prefix = [rng.choice([0, 31, 128, 129, 500, rng.randint(1, 1500)]) for _ in range(n)]
    lens = []
    for s, P in zip(sizes, prefix):
        lens += [P + rng.choice([0, Sq, Sq, 130, rng.randint(Sq, 300), rng.randint(Sq, 700)]) for _ in range(s)]
    D, page = rng.choice([64, 128]), rng.choice([32, 64, 96, 128])
    dtype = rng.choice([torch.bfloat16, torch.float16])
    check(fa, inputs(Hq, Hkv, D, page, starts, prefix, lens, Sq, dtype, seed=seed), D ** -0.5)


def test_many_groups_and_sequences(fa):
    """More groups and sequences than a block has threads."""
    rng = random.Random(1)
    starts, lens, prefix = [0], [], []
    for i in range(400):
        n = rng.choice([1, 1, 2, 3])
        P = rng.choice([0, 20, 33, 64])
        starts.append(starts[-1] + n)
        prefix.append(P)
        lens += [P + rng.choice([0, 1, 2, 40]) for _ in range(n)]
    check(fa, inputs(2, 1, 64, 32, starts, prefix, lens, 1, torch.bfloat16, seed=7), 0.125)


@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0])
def test_scales(fa, scale):
    check(fa, inputs(8, 2, 64, 32, [0, 5], [200], [210, 230, 201, 400, 200], 1, torch.bfloat16, seed=2), scale)


def test_scores_that_jump(fa):
    """Keys far larger in the middle of the prefix: rows renew their maximum there."""
    t = inputs(16, 1, 64, 32, [0, 9], [900], [950 + i for i in range(9)], 1, torch.float16, seed=6)
    t[1][t[3][0, 14].long()] *= 40
    check(fa, t, 0.125)


def test_bad_starts_share_nothing_and_are_reported(fa):
    full = inputs(4, 2, 64, 32, [0, 0], [0], [100, 170, 40], 1, torch.bfloat16, seed=9)
    for starts in ([1, 0], [0, 4], [-1, 2], [0, 2, 1]):
        t = full[:5] + (torch.tensor(starts, dtype=torch.int32),
                        torch.tensor([90] * (len(starts) - 1), dtype=torch.int32))
        out, lse = run(fa, t, 0.125, fa.FA_ERR_BOUNDS)
        q, kp, vp, table, lens = full[:5]
        sp.check_decode(out, lse, q, kp, vp, table.numpy(), lens.tolist(), 0.125)
    assert fa.fa_device_error()[0] == fa.FA_OK


@pytest.mark.parametrize("P", [-1, 193, 2 ** 31 - 1])
def test_bad_prefix_lengths_count_as_0_and_are_reported(fa, P):
    full = inputs(4, 2, 64, 32, [0, 0], [0], [100, 170, 40], 1, torch.bfloat16, seed=10)
    t = full[:5] + (torch.tensor([0, 3], dtype=torch.int32), torch.tensor([P], dtype=torch.int32))
    out, lse = run(fa, t, 0.125, fa.FA_ERR_BOUNDS)
    q, kp, vp, table, lens = full[:5]
    sp.check_decode(out, lse, q, kp, vp, table.numpy(), lens.tolist(), 0.125)


def test_bad_pages_mask_their_keys_and_are_reported(fa):
    t = inputs(8, 2, 64, 32, [0, 3], [200], [230, 260, 300], 1, torch.bfloat16, seed=11)
    t[3][0, 2] = -1          # of the prefix: masked for the whole group
    t[3][1:, 2] = -1
    t[3][2, 7] = 10 ** 7     # of one sequence's own
    out, lse = run(fa, t, 0.125, fa.FA_ERR_BOUNDS)
    q, kp, vp, table, lens = t[:5]
    k2, v2 = kp.clone(), vp.clone()
    full = table.clone()
    for b in (1, 2):  # the end of the prefix through the first row, as the kernel reads it
        k2[table[b, 6].long(), :8] = kp[table[0, 6].long(), :8]
        v2[table[b, 6].long(), :8] = vp[table[0, 6].long(), :8]
    sp.check_decode(out, lse, q, k2, v2, full.numpy(), lens.tolist(), 0.125)
    assert fa.fa_device_error()[0] == fa.FA_OK


def test_every_page_bad(fa):
    t = inputs(4, 1, 128, 64, [0, 2], [64], [100, 70], 1, torch.bfloat16, seed=4)
    t[3][:] = -1
    out, lse = run(fa, t, 0.1, fa.FA_ERR_BOUNDS)
    assert not out.any() and torch.isneginf(lse).all()


def test_lengths_past_the_table_are_clamped(fa):
    """As in the paged decode."""
    t = list(inputs(4, 2, 64, 32, [0, 2], [64], [96, 96, 96], 1, torch.bfloat16, seed=12))
    ref = run(fa, t, 0.125)
    t[4] = torch.tensor([97, 2 ** 31 - 1, 96], dtype=torch.int32)
    out = run(fa, t, 0.125)
    assert torch.equal(out[0], ref[0]) and torch.equal(out[1], ref[1])
    t[4] = torch.tensor([-5, 96, 0], dtype=torch.int32)
    out, lse = run(fa, t, 0.125)
    assert not out[0].any() and not out[2].any() and torch.isneginf(lse[0]).all()


def test_cache_without_pages(fa):
    t = list(inputs(4, 2, 64, 32, [0, 3], [0], [0, 0, 0], 1, torch.bfloat16, seed=5, width=1))
    t[3] = t[3][:, :0].contiguous()
    out, lse = run(fa, t, 0.125)
    assert not out.any() and torch.isneginf(lse).all()


def test_rows_with_a_score_that_is_nan(fa):
    t = inputs(4, 2, 64, 64, [0, 3], [300], [320, 900, 301], 1, torch.bfloat16, seed=13)
    sound = run(fa, t, 0.125)
    t[0][1, 0, 2, 5] = float("nan")
    out, lse = run(fa, t, 0.125)
    want = torch.zeros(3, 1, 4, dtype=torch.bool)
    want[1, 0, 2] = True
    assert torch.equal(torch.isnan(lse.cpu()), want)
    assert torch.equal(torch.isnan(out.cpu()), want[..., None].expand(out.shape))
    keep = ~want.cuda()
    assert torch.equal(out[keep], sound[0][keep]) and torch.equal(lse[keep], sound[1][keep])


@pytest.mark.parametrize("Hq,Hkv,D,B,P,own,page", [(64, 8, 128, 40, 20000, 700, 64), (8, 2, 64, 5, 65536, 4000, 128),
                                                   (128, 8, 128, 20, 9000, 300, 32)])
def test_long_prefixes_against_the_paged_decode(fa, Hq, Hkv, D, B, P, own, page):
    """Both within their bounds of the same rows: their difference is within the sum."""
    rng = random.Random(P)
    g = torch.Generator(device="cuda").manual_seed(P)
    lens = [P + rng.randint(1, own) for _ in range(B)]
    whole_pages, used = P // page, P // page
    rows = []
    for L in lens:
        more = -(-L // page) - whole_pages
        rows.append(list(range(whole_pages)) + list(range(used, used + more)))
        used += more
    width = max(len(r) for r in rows)
    kp = torch.randn(used, page, Hkv, D, generator=g, device="cuda").bfloat16()
    vp = torch.randn(used, page, Hkv, D, generator=g, device="cuda").bfloat16()
    r = P % page
    for row in rows[1:]:
        kp[row[whole_pages], :r] = kp[rows[0][whole_pages], :r]
        vp[row[whole_pages], :r] = vp[rows[0][whole_pages], :r]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    table, lens = i32([x + [0] * (width - len(x)) for x in rows]), i32(lens)
    q = torch.randn(B, 1, Hq, D, generator=g, device="cuda").bfloat16()
    a, la = fa.decode_paged(q, kp, vp, table, lens, D ** -0.5, lse=True)
    b, lb = fa.decode_shared(q, kp, vp, table, lens, i32([0, B]), i32([P]), D ** -0.5, lse=True)
    again = fa.decode_shared(q, kp, vp, table, lens, i32([0, B]), i32([P]), D ** -0.5)
    torch.cuda.synchronize()
    assert fa.fa_device_error()[0] == fa.FA_OK
    assert torch.equal(b, again)
    # Each O: P's rounding 2^-8 of sum p |v| / sum p (below 1 here: |v| is 0.8 on average,
    # and so many keys share the weight), one rounding of O.
    assert ((a.double() - b.double()).abs() <= 2 * 2.0 ** -8 * (1.0 + a.double().abs()) * 1.02).all()
    assert ((la - lb).abs() <= 2 * (132 * 2.0 ** -24 * 0.125 * 400 + 2.0 ** -18)).all()
