"""Verification of drafted trees (fa_verify_tree) against a plain 64-bit walk:
the answers are whole numbers and have to be equal."""
import random

import numpy as np
import pytest
import torch

from tests import tree_plain as tp

pytestmark = pytest.mark.gpu


def inputs(B, N, V, draft, chain, seed, sharp=2.5):
    rng = random.Random(seed)
    g = torch.Generator().manual_seed(seed)
    parents = [[s - 1 for s in range(N)]] * B if chain else tp.random_parents(B, N, rng, 0.05)
    logits = torch.randn(B, N, V, generator=g) * sharp
    p = torch.softmax(logits, -1)
    q = torch.softmax(logits * 0.9 + 0.4 * torch.randn(B, N, V, generator=g), -1)
    tokens = torch.zeros(B, N, dtype=torch.int32)
    for b in range(B):
        for s in range(1, N):
            at = max(parents[b][s], 0)
            tokens[b, s] = int(torch.multinomial((q if draft else p)[b, at], 1, generator=g))
    u = torch.rand(B, N, generator=g)
    return p, q if draft else None, tokens, torch.tensor(parents, dtype=torch.int32), u


def check(fa, p, q, tokens, parents, u, status=None):
    path, count, nxt = fa.verify_tree(p.cuda(), None if q is None else q.cuda(), tokens.cuda(),
                                      parents.cuda(), u.cuda())
    torch.cuda.synchronize()
    st, detail = fa.fa_device_error()
    assert st == (fa.FA_OK if status is None else status), hex(detail)
    N = p.shape[1]
    for b in range(p.shape[0]):
        way, tok = tp.verify(p[b].numpy(), None if q is None else q[b].numpy(), tokens[b].tolist(),
                             parents[b].tolist(), u[b].tolist())
        assert path[b].tolist() == way + [-1] * (N - len(way)), b
        assert int(count[b]) == len(way) and int(nxt[b]) == tok, b
    return path, count, nxt


@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("B,N,V,chain", [
    (1, 1, 1, True), (3, 1, 1001, True), (4, 5, 32000, True), (6, 9, 37, False),
    (2, 64, 5003, False), (20, 16, 640, False), (2, 33, 128256, False), (3, 64, 130, True),
])
def test_verify(fa, B, N, V, chain, draft):
    check(fa, *inputs(B, N, V, draft, chain, seed=B + N + V))


def test_many_rejected_siblings(fa):
    """All nodes children of the root and drafted from a poor distribution:
    many residuals, one after another."""
    B, N, V = 8, 24, 2000
    p, q, tokens, parents, u = inputs(B, N, V, True, False, seed=7)
    parents[:, 1:] = 0
    q = torch.softmax(torch.randn(B, N, V, generator=torch.Generator().manual_seed(8)), -1)
    tokens = torch.randint(0, V, (B, N), generator=torch.Generator().manual_seed(9)).int()
    check(fa, p, q, tokens, parents, u)


@pytest.mark.parametrize("draft", [True, False])
def test_repeated_sibling_tokens(fa, draft):
    """The same token twice under one node: after its rejection it is never
    accepted there."""
    p, q, tokens, parents, u = inputs(6, 8, 300, draft, False, seed=3)
    parents[:, 1:] = 0
    tokens[:, 2:] = tokens[:, 1:2]
    u[:, 1:] = 0.9999
    path, count, nxt = check(fa, p, q, tokens, parents, u)


def test_borders(fa):
    """Uniform probabilities of 1/8, u on the borders: the border belongs to
    the token above it; u = 0 accepts anything with mass, and draws the first
    token with mass."""
    V = 8
    u0 = torch.tensor([0.0, 0.125, 0.25 - 2.0 ** -26, 0.5, 0.875, 1 - 2.0 ** -24])
    B = len(u0)
    p = torch.full((B, 1, V), 0.125)
    p[:, :, 0] = 0.0
    p[:, :, 1] = 0.25
    tokens = torch.zeros(B, 1, dtype=torch.int32)
    parents = torch.full((B, 1), -1, dtype=torch.int32)
    _, _, nxt = check(fa, p, None, tokens, parents, u0[:, None].contiguous())
    assert nxt.tolist() == [1, 1, 1, 4, 7, 7]


def test_rows_without_mass_and_values_that_are_no_probabilities(fa):
    p, q, tokens, parents, u = inputs(6, 4, 50, True, True, seed=5)
    p[0, 0] = 0.0                       # nothing at the root
    p[1, 0] = float("nan")
    q[2, 0] = p[2, 0]                   # residual zero after a rejection: impossible but for u = 1
    u[2, 1] = 1.0
    p[3, 0, ::2] = -0.5
    p[3, 0, 1] = float("inf")
    q[4, 0] = float("inf")
    q[5, :, 7] = float("nan")
    path, count, nxt = check(fa, p, q, tokens, parents, u)
    assert int(nxt[0]) == -1 and int(nxt[1]) == -1


def test_last_token_when_u_is_one(fa):
    p, q, tokens, parents, u = inputs(3, 1, 700, False, True, seed=6)
    u[:] = 1.0
    check(fa, p, q, tokens, parents, u)


def test_bad_nodes_are_unreachable_and_reported(fa):
    p, q, tokens, parents, u = inputs(3, 6, 64, True, True, seed=4)
    u[:, 1:] = 0.0
    tokens[0, 2] = 64
    tokens[1, 1] = -1
    parents[2, 3] = 5
    path, count, _ = check(fa, p, q, tokens, parents, u, status=fa.FA_ERR_BOUNDS)
    assert count.tolist() == [2, 1, 3]
    assert fa.fa_device_error()[0] == fa.FA_OK


def test_unaligned_rows(fa):
    """Probabilities at an address that is a multiple of 4 bytes only."""
    p, q, tokens, parents, u = inputs(2, 5, 1000, True, False, seed=2)
    def shift(t):
        flat = torch.empty(t.numel() + 1, device="cuda")
        flat[1:] = t.reshape(-1).cuda()
        return flat[1:].view(t.shape)
    a = fa.verify_tree(shift(p), shift(q), tokens.cuda(), parents.cuda(), u.cuda())
    b = fa.verify_tree(p.cuda(), q.cuda(), tokens.cuda(), parents.cuda(), u.cuda())
    for x, y in zip(a, b):
        assert torch.equal(x, y)


def test_accepted_share_follows_the_target(fa):
    """Two drafts per node over many seeds: tokens come out with the target's
    frequencies.  With n = 4096 draws a frequency of probability f is off by
    more than 5 sqrt(f (1 - f) / n) about once in two million."""
    n, V = 4096, 6
    g = torch.Generator().manual_seed(1)
    f = torch.softmax(torch.randn(V, generator=g), -1)
    d = torch.softmax(torch.randn(V, generator=g), -1)
    p = f.expand(n, 3, V).contiguous()
    q = d.expand(n, 3, V).contiguous()
    parents = torch.tensor([[-1, 0, 0]] * n, dtype=torch.int32)
    tokens = torch.multinomial(d.expand(n, V), 3, replacement=True, generator=g).int()
    u = torch.rand(n, 3, generator=g)
    path, count, nxt = fa.verify_tree(p.cuda(), q.cuda(), tokens.cuda(), parents.cuda(), u.cuda())
    first = torch.where(count.cpu() > 1, tokens.gather(1, path[:, 1:2].cpu().clamp(min=0).long())[:, 0],
                        nxt.cpu())
    share = np.bincount(first.numpy(), minlength=V) / n
    ff = f.double().numpy()
    assert np.all(np.abs(share - ff) <= 5 * np.sqrt(ff * (1 - ff) / n))


@pytest.mark.parametrize("closeness", [1e-2, 1e-3, 1e-5])
@pytest.mark.parametrize("V", [500, 32001, 128000])
def test_rejections_of_a_draft_close_to_the_target(fa, V, closeness):
    """Residuals with little mass left, several rejections deep: the children are
    tokens that the draft makes too likely, whose residual is zero.  With masses
    from 1e-2 down to 1e-5 borders are good to about 1e-9, and no u lies so close to
    one."""
    B, N = 6, 6
    g = torch.Generator().manual_seed(V)
    logits = torch.randn(B, N, V, generator=g) * 1.5
    p = torch.softmax(logits, -1)
    q = torch.softmax(logits + closeness * torch.randn(B, N, V, generator=g), -1)
    parents = torch.zeros(B, N, dtype=torch.int32)
    parents[:, 4:] = 3  # (reached only where node 3 is accepted)
    tokens = torch.zeros(B, N, dtype=torch.int32)
    u = torch.rand(B, N, generator=g)
    u[:, 1:4] = 1 - 2.0 ** -24
    for b in range(B):
        over = torch.nonzero(q[b, 0] > p[b, 0] * (1 + 1e-6))[:, 0]
        tokens[b, 1:4] = over[torch.randint(0, len(over), (3,), generator=g)].int()
        if b % 2:  # the third by a residual of its own: accepted or not
            under = torch.nonzero(q[b, 0] < p[b, 0])[:, 0]
            tokens[b, 3] = int(under[torch.randint(0, len(under), (1,), generator=g)])
            u[b, 3] = torch.rand(1, generator=g)
            tokens[b, 4:] = tokens[b, 1:3]
    path, count, _ = check(fa, p, q, tokens, parents, u)
    assert (count[::2] == 1).all()  # three rejections
