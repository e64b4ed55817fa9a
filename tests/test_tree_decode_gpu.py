"""Attention of drafted trees over a paged cache (fa_decode_tree_fwd) against a
plain 64-bit form: sizes around the tile and page edges, row counts around one
and two row tiles, trees of one node to 64, chains, forests, unused nodes,
padding, NaN wherever nothing may be read, bad pages."""
import math
import random

import pytest
import torch

from tests import tree_plain as tp

pytestmark = pytest.mark.gpu


def inputs(B, N, Hq, Hkv, D, page, lens, dtype, seed, max_pages=None, parents=None, unused=0.0):
    """Shuffled pages; every slot that holds no token is NaN, and so are the
    slots of unused nodes."""
    rng = random.Random(seed)
    g = torch.Generator().manual_seed(seed)
    max_pages = max_pages or max(1, -(-max(max(lens), 1) // page))
    num_pages = B * max_pages + 3
    kp = torch.full((num_pages, page, Hkv, D), float("nan"), dtype=dtype)
    vp = kp.clone()
    table = torch.randperm(num_pages, generator=g)[:B * max_pages].reshape(B, max_pages).int()
    parents = parents or tp.random_parents(B, N, rng, unused)
    for b, L in enumerate(lens):
        for t in range(min(L, max_pages * page)):
            pid = int(table[b, t // page])
            kp[pid, t % page] = torch.randn(Hkv, D, generator=g).to(dtype)
            vp[pid, t % page] = torch.randn(Hkv, D, generator=g).to(dtype)
        if L >= N and L <= max_pages * page:
            usable = tp.tree_sees(parents[b], N)[1]
            for s in range(N):
                if not usable[s]:
                    t = L - N + s
                    kp[int(table[b, t // page]), t % page] = float("nan")
                    vp[int(table[b, t // page]), t % page] = float("nan")
    q = torch.randn(B, N, Hq, D, generator=g).to(dtype)
    return (q, kp, vp, table, torch.tensor(lens, dtype=torch.int32),
            torch.tensor(parents, dtype=torch.int32))


def run(fa, t, scale, status=None):
    out, lse = fa.decode_tree(*(x.cuda() for x in t), scale, lse=True)
    torch.cuda.synchronize()
    st, detail = fa.fa_device_error()
    assert st == (fa.FA_OK if status is None else status), hex(detail)
    return out, lse


def check(fa, t, scale, status=None):
    out, lse = run(fa, t, scale, status)
    q, kp, vp, table, lens, parents = t
    tp.check_tree(out, lse, q, kp, vp, table.numpy(), lens.tolist(), parents.tolist(), scale)
    return out, lse


@pytest.mark.parametrize("B,N,Hq,Hkv,D,page,lens,dtype", [
    (1, 1, 2, 1, 64, 32, [1], torch.bfloat16),               # one token, one key
    (1, 1, 8, 2, 128, 64, [129], torch.float16),             # a key past the first tile
    (1, 7, 6, 2, 128, 96, [385], torch.bfloat16),            # odd group, pages inside tiles
    (2, 16, 8, 1, 64, 64, [128, 300], torch.float16),        # 128 rows: one full row tile
    (1, 43, 3, 1, 128, 128, [515], torch.bfloat16),          # 129 rows: a second tile of one row
    (2, 64, 4, 1, 128, 32, [64, 700], torch.bfloat16),       # 256 rows; a tree without a prompt
    (1, 64, 5, 1, 64, 256, [257], torch.float16),            # 320 rows: three CTAs per unit
    (1, 56, 16, 1, 128, 64, [700], torch.bfloat16),          # 896 rows: four CTAs, half of the last
    (2, 61, 27, 3, 64, 64, [400, 61], torch.float16),        # 549 rows: five CTAs, one row tile each
    (3, 5, 16, 16, 64, 32, [5, 260, 131], torch.bfloat16),   # MHA
    (1, 64, 16, 1, 128, 64, [900], torch.bfloat16),          # 1024 rows, MQA
    (2, 33, 4, 4, 128, 128, [161, 1100], torch.float16),
])
def test_tree_decode(fa, B, N, Hq, Hkv, D, page, lens, dtype):
    t = inputs(B, N, Hq, Hkv, D, page, lens, dtype, seed=N + D + Hq)
    check(fa, t, 1 / math.sqrt(D))


@pytest.mark.parametrize("B,Hq,Hkv", [(40, 4, 2), (200, 2, 1)])
def test_ragged_batches_with_padding(fa, B, Hq, Hkv):
    """More sequences than a warp's lanes and than the SMs; empty and short
    sequences among them; ranges that hold several whole sequences."""
    rng = random.Random(B)
    lens = [rng.choice([0, 3, 6, 7, 64, 127, 128, 129, rng.randint(7, 400)]) for _ in range(B)]
    check(fa, inputs(B, 6, Hq, Hkv, 64, 32, lens, torch.bfloat16, seed=B), 0.125)


@pytest.mark.parametrize("seed", range(5))
def test_shares_that_end_anywhere(fa, seed):
    """Short and long sequences side by side: shares of the list that begin and
    end in the middle of units, between them, and in none."""
    rng = random.Random(100 + seed)
    B, N, Hkv = rng.choice([7, 31, 33, 60]), rng.randint(1, 5), rng.choice([1, 2, 5])
    Hq = Hkv * rng.choice([1, 3, 60])
    if Hq > 60:
        B = 7
    lens = [rng.choice([0, N, 128, 129, 500, rng.randint(N, 700), rng.randint(N, 2600)]) for _ in range(B)]
    check(fa, inputs(B, N, Hq, Hkv, 64, 64, lens, torch.bfloat16, seed=seed), 0.125)


def test_every_sequence_is_padding(fa):
    t = inputs(3, 4, 4, 2, 64, 32, [0, 3, 2], torch.bfloat16, seed=5, max_pages=2)
    out, lse = check(fa, t, 0.125)
    assert not out.any() and torch.isneginf(lse).all()


def test_unused_nodes_and_nodes_below_them(fa):
    par = [[-1, 0, -2, 2, 1, 3, -1, 6], [-2, 0, -1, 2, -2, 3, 4, -2]]
    t = inputs(2, 8, 4, 2, 128, 64, [200, 60], torch.bfloat16, seed=8, parents=par)
    out, lse = check(fa, t, 0.09)
    for b, s in ((0, 2), (0, 3), (0, 5), (1, 0), (1, 1), (1, 6), (1, 7)):
        assert not out[b, s].any() and torch.isneginf(lse[b, s]).all()


def test_random_unused_nodes(fa):
    check(fa, inputs(2, 40, 4, 1, 64, 32, [140, 333], torch.float16, seed=3, unused=0.2), 0.125)


@pytest.mark.parametrize("scale", [0.0, -0.1, 1.5])
def test_scales(fa, scale):
    """No scores, the sign reversed, and scores of tens of units (the running
    maximum has to be renewed)."""
    check(fa, inputs(1, 9, 4, 1, 64, 64, [700], torch.bfloat16, seed=2), scale)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_growing_scores_renew_the_maximum(fa, dtype):
    """Keys that grow along the cache: every tile's scores exceed the last
    one's by tens of units, up to the tree."""
    t = inputs(1, 12, 2, 1, 64, 64, [1000], dtype, seed=6)
    q, kp, vp, table, lens, parents = t
    for i in range(table.shape[1]):
        kp[int(table[0, i])] *= 0.25 * (1 + i // 2)
    check(fa, t, 1.0)


def test_chain_gives_paged_decode(fa):
    """parents[s] = s - 1 is the causal order of fa_decode_paged_fwd: both
    within bounds of the same 64-bit values."""
    N = 5
    t = inputs(2, N, 8, 2, 128, 64, [700, 61], torch.bfloat16, seed=1,
               parents=[[s - 1 for s in range(N)]] * 2)
    out, lse = check(fa, t, 0.088)
    q, kp, vp, table, lens, parents = t
    o2, l2 = fa.decode_paged(*(x.cuda() for x in (q, kp, vp, table, lens)), 0.088, lse=True)
    torch.cuda.synchronize()
    assert (out.float() - o2.float()).abs().max().item() <= 2 * 2.0 ** -8 * o2.float().abs().max().item()
    assert (lse - l2).abs().max().item() <= 2.0 ** -18


def test_bad_parents_pages_and_lengths_are_reported(fa):
    t = list(inputs(3, 6, 4, 2, 64, 32, [100, 90, 40], torch.bfloat16, seed=9, max_pages=4))
    t[5][0, 3] = 3        # its own parent
    t[5][0, 4] = 77
    t[5][1, 2] = -9
    t[3][1, 1] = 10 ** 6  # a page that does not exist: its keys are masked
    t[4][2] = 129         # past the page table: padding
    q, kp, vp, table, lens, parents = t
    for b, s in ((0, 3), (0, 4), (1, 2)):  # what a bad node's slot holds is not read
        L = int(lens[b])
        slot = L - 6 + s
        vp[int(table[b, slot // 32]), slot % 32] = float("nan")
    check(fa, tuple(t), 0.125, status=fa.FA_ERR_BOUNDS)
    assert fa.fa_device_error()[0] == fa.FA_OK


def test_page_that_is_bad_everywhere(fa):
    """Every key masked: O = 0, log-sum-exp -inf; nothing hangs."""
    t = inputs(1, 3, 4, 1, 128, 64, [64], torch.bfloat16, seed=4)
    t[3][0, 0] = -1
    out, lse = run(fa, t, 0.1, fa.FA_ERR_BOUNDS)
    assert not out.any() and torch.isneginf(lse).all()


def test_other_stream_and_preallocated_outputs(fa):
    t = tuple(x.cuda() for x in inputs(2, 8, 8, 2, 128, 64, [300, 77], torch.bfloat16, seed=11))
    ref, ref_lse = fa.decode_tree(*t, 0.088, lse=True)
    out, lse = torch.empty_like(ref), torch.empty_like(ref_lse)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    fa.decode_tree(*t, 0.088, out=out, lse=lse, stream=side)
    fresh = fa.decode_tree(*t, 0.088, stream=side)
    side.synchronize()
    assert torch.equal(out, ref) and torch.equal(lse, ref_lse) and torch.equal(fresh, ref)
    assert fa.fa_device_error()[0] == fa.FA_OK


def test_many_rows_long_context(fa):
    """Several CTAs per unit over a long cache, split inside it: against the
    same operator run on one node at a time, each a chain of its ancestors."""
    B, N, Hq, Hkv, D, L = 1, 24, 32, 2, 128, 20000
    g = torch.Generator(device="cuda").manual_seed(0)
    page, P = 128, -(-L // 128)
    kp = torch.randn(P, page, Hkv, D, generator=g, device="cuda").bfloat16()
    vp = torch.randn(P, page, Hkv, D, generator=g, device="cuda").bfloat16()
    q = torch.randn(B, N, Hq, D, generator=g, device="cuda").bfloat16()
    table = torch.arange(P, dtype=torch.int32, device="cuda")[None]
    lens = torch.tensor([L], dtype=torch.int32, device="cuda")
    parents = torch.tensor(tp.random_parents(1, N, random.Random(4)), dtype=torch.int32)
    out, lse = fa.decode_tree(q, kp, vp, table, lens, parents.cuda(), D ** -0.5, lse=True)
    torch.cuda.synchronize()
    assert fa.fa_device_error()[0] == fa.FA_OK
    see = torch.from_numpy(tp.tree_sees(parents[0].tolist(), N)[0])
    ok = torch.ones(N, L, dtype=torch.bool)
    ok[:, L - N:] = see
    ok = ok.cuda()
    k = kp.reshape(-1, Hkv, D)[:L].double()
    v = vp.reshape(-1, Hkv, D)[:L].double()
    for h in (0, 9, 16, 31):
        s = q[0, :, h].double() @ k[:, h // 16].T * D ** -0.5
        s = torch.where(ok, s, -math.inf)
        z = torch.logsumexp(s, -1)
        p = torch.exp(s - z[:, None])
        ref = p @ v[:, h // 16]
        size = p @ v[:, h // 16].abs()
        # As check_tree: E <= 132 * 2^-24 * scale * sum |q k| with the sum below 400.
        tol = 2.0 ** -8 * (size + ref.abs()) * 1.01 + 2 * (132 * tp.U32 * 0.0885 * 400 + 2.0 ** -21) * size
        assert ((out[0, :, h].double() - ref).abs() <= tol).all()
        assert ((lse[0, :, h].double() - z).abs() <= 132 * tp.U32 * 0.0885 * 400 + 2.0 ** -18).all()


@pytest.mark.parametrize("lens,bad", [([0, 0, 0], False), ([0, -4, 0], False), ([0, 9, 0], True),
                                      ([2, 0, 0], True)])
def test_cache_without_pages(fa, lens, bad):
    """max_pages 0: every sequence is padding, and a length above 0 is past the
    page table, as with pages."""
    t = list(inputs(3, 4, 4, 2, 64, 32, [0, 0, 0], torch.bfloat16, seed=5, max_pages=1))
    t[3] = t[3][:, :0].contiguous()
    t[4] = torch.tensor(lens, dtype=torch.int32)
    out, lse = run(fa, t, 0.125, fa.FA_ERR_BOUNDS if bad else None)
    assert not out.any() and torch.isneginf(lse).all()
    assert fa.fa_device_error()[0] == fa.FA_OK


@pytest.mark.parametrize("N,Hq,Hkv,lens", [(6, 4, 2, [90, 41]), (6, 4, 2, [2600, 41]), (64, 4, 1, [700, 64])])
def test_rows_with_a_score_that_is_nan(fa, N, Hq, Hkv, lens):
    """NaN in q, or in the K of a node: O and log-sum-exp of the rows that have
    such a score are NaN (not those of a row without keys), the others as ever."""
    t = inputs(2, N, Hq, Hkv, 64, 64, lens, torch.bfloat16, seed=N)
    q, kp, vp, table, lens, parents = t
    q[0, 1, 2, 5] = float("nan")
    at = lens[1].item() - N + 2
    kp[int(table[1, at // 64]), at % 64, 0, 3] = float("nan")
    out, lse = run(fa, t, 0.125)
    want = torch.zeros(2, N, Hq, dtype=torch.bool)
    want[0, 1, 2] = True
    see = tp.tree_sees(parents[1].tolist(), N)[0][:, 2]
    want[1, torch.from_numpy(see), :Hq // Hkv] = True
    assert torch.equal(torch.isnan(lse.cpu()), want)
    assert torch.equal(torch.isnan(out.cpu()), want[..., None].expand(out.shape))
    sound = [x.clone() for x in t]
    sound[0].nan_to_num_(0.0)
    sound[1].nan_to_num_(0.0)
    o2, l2 = run(fa, sound, 0.125)
    keep = ~want.cuda()
    assert torch.equal(out[keep], o2[keep]) and torch.equal(lse[keep], l2[keep])
