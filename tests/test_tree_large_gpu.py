"""Offsets past 2^31 elements: caches, head rows and probabilities whose last
rows lie beyond what a 32-bit index reaches."""
import random

import numpy as np
import pytest
import torch

from tests import tree_plain as tp

pytestmark = pytest.mark.gpu


def test_cache_past_2_31_elements(fa):
    """Append, attend and compact in the last pages of a pool of 2.2e9 elements."""
    B, N, Hq, Hkv, D, page, P = 2, 6, 8, 8, 128, 64, 33600
    assert P * page * Hkv * D > 2 ** 31
    kp = torch.zeros(P, page, Hkv, D, dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    lens = [150, 77]
    table = torch.tensor([[P - 1, P - 3, P - 2], [P - 5, P - 4, 0]], dtype=torch.int32)
    g = torch.Generator().manual_seed(1)
    for b, L in enumerate(lens):
        for i in range(-(-L // page)):
            kp[int(table[b, i])] = torch.randn(page, Hkv, D, generator=g).bfloat16().cuda()
            vp[int(table[b, i])] = torch.randn(page, Hkv, D, generator=g).bfloat16().cuda()
    qkv = torch.randn(B, N, Hq + 2 * Hkv, D, generator=g).bfloat16().cuda()
    w = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    f = (10000.0 ** (-torch.arange(64, dtype=torch.float64) / 64)).float()
    ld, td = torch.tensor(lens, dtype=torch.int32).cuda(), table.cuda()
    q = fa.qk_norm_rope_append(qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:], w, w,
                               f.cuda(), kp, vp, td, ld, 1e-6)
    torch.cuda.synchronize()
    for b, L in enumerate(lens):
        for s in range(N):
            t = L - N + s
            pid = int(table[b, t // page])
            assert torch.equal(vp[pid, t % page], qkv[b, s, Hq + Hkv:])
            tp.check_rope(kp[pid, t % page][None], qkv[b, s, Hq:Hq + Hkv][None], w,
                          tp.angles([t], f), 1e-6, False)
    parents = torch.tensor(tp.random_parents(B, N, random.Random(2)), dtype=torch.int32)
    out, lse = fa.decode_tree(q, kp, vp, td, ld, parents.cuda(), 0.09, lse=True)
    torch.cuda.synchronize()
    # The same pages in a small pool.
    small = torch.full_like(table, 0)
    ks, vs = [kp[0].cpu()], [vp[0].cpu()]
    for b in range(B):
        for i in range(3):
            small[b, i] = len(ks)
            ks.append(kp[int(table[b, i])].cpu())
            vs.append(vp[int(table[b, i])].cpu())
    tp.check_tree(out, lse, q.cpu(), torch.stack(ks), torch.stack(vs), small.numpy(), lens,
                  parents.tolist(), 0.09)
    path = torch.tensor([[0, 2, 5, -1, -1, -1], [0, 1, 3, 4, -1, -1]], dtype=torch.int32)
    count = torch.tensor([3, 4], dtype=torch.int32)
    new = fa.compact_tree(kp, vp, td, ld, path.cuda(), count.cuda())
    torch.cuda.synchronize()
    for was, pool in ((ks, kp), (vs, vp)):
        want = torch.stack(was)[None].clone()
        assert new.tolist() == tp.compact(want, small.numpy(), lens, path.tolist(), count.tolist(), N)
        for b in range(B):
            for i in range(3):
                if int(table[b, i]):
                    assert torch.equal(pool[int(table[b, i])].cpu(), want[0, int(small[b, i])])
    assert fa.fa_device_error()[0] == fa.FA_OK


def test_layers_past_2_31_elements(fa):
    """The last layer of a pool of 2.2e9 elements is compacted too."""
    layers, P, page, Hkv, D, N = 70, 30, 64, 128, 128, 4
    assert layers * P * page * Hkv * D > 2 ** 31
    kp = torch.zeros(layers, P, page, Hkv, D, dtype=torch.float16, device="cuda")
    vp = torch.zeros_like(kp)
    rows = torch.arange(1, N + 1, device="cuda").half()
    kp[:, 29, 60:] = rows[:, None, None]
    vp[:, 29, 60:] = -rows[:, None, None]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    new = fa.compact_tree(kp, vp, i32([[29]]), i32([64]), i32([[1, 3, -1, -1]]), i32([2]))
    torch.cuda.synchronize()
    assert new.tolist() == [62] and fa.fa_device_error()[0] == fa.FA_OK
    for layer in (0, 35, layers - 1):
        for pool, sign in ((kp, 1), (vp, -1)):
            assert (pool[layer, 29, 60] == 2 * sign).all() and (pool[layer, 29, 61] == 4 * sign).all()
            assert (pool[layer, 29, 62] == 3 * sign).all() and (pool[layer, 29, 63] == 4 * sign).all()


@pytest.mark.parametrize("T,Hq,Hkv,D", [(135000, 128, 8, 128), (8500001, 4, 2, 64)])
def test_heads_past_2_31_elements(fa, T, Hq, Hkv, D):
    """The last tokens, forward and gradient: a token in several steps, and
    several tokens in one."""
    assert T * Hq * D > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(3)
    qkv = torch.empty(T, Hq + Hkv, D, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    q, k = qkv[:, :Hq], qkv[:, Hq:]
    w = torch.empty(D, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    f = (10000.0 ** (-torch.arange(D // 2, dtype=torch.float64) / (D // 2))).float()
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    qo, ko = fa.qk_norm_rope(q, k, w, w, f.cuda(), pos, 1e-6)
    at = [0, 65535, 131071, 131072, T - 1]
    ang = tp.angles(at, f)
    tp.check_rope(qo[at], q[at], w, ang, 1e-6, False)
    tp.check_rope(ko[at], k[at], w, ang, 1e-6, False)
    dq, dk, _, _ = fa.qk_norm_rope_backward(qo, ko, q, k, w, w, f.cuda(), pos, 1e-6)
    torch.cuda.synchronize()
    for x, gr, dx in ((q, qo, dq), (k, ko, dk)):
        ref, _, size, _ = tp.norm_rope_grad(x[at], w, gr[at], ang, 1e-6, False)
        assert np.all(np.abs(tp.f64(dx[at]) - ref) <= 2.0 ** -8 * np.abs(ref) + 97 * tp.U32 * size)
    assert fa.fa_device_error()[0] == fa.FA_OK


def test_probabilities_past_2_31(fa):
    """The last sequences of 2.3e9 probabilities."""
    B, N, V = 72, 64, 500000
    assert B * N * V > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(4)
    p = torch.empty(B, N, V, device="cuda").exponential_(generator=g).div_(V)
    parents = torch.tensor(tp.random_parents(B, N, random.Random(5)), dtype=torch.int32)
    tokens = torch.randint(0, V, (B, N), generator=torch.Generator().manual_seed(6)).int()
    u = torch.rand(B, N, generator=torch.Generator().manual_seed(7))
    u[:, 1::2] = 0.0  # half of the nodes accepted where they are reached
    path, count, nxt = fa.verify_tree(p, None, tokens.cuda(), parents.cuda(), u.cuda())
    torch.cuda.synchronize()
    assert fa.fa_device_error()[0] == fa.FA_OK
    for b in (0, 40, 67, 68, B - 1):
        way, tok = tp.verify(p[b].cpu().numpy(), None, tokens[b].tolist(), parents[b].tolist(),
                             u[b].tolist())
        assert path[b].tolist() == way + [-1] * (N - len(way)) and int(nxt[b]) == tok


def test_length_close_to_2_31(fa):
    """The longest lengths, whose last tile ends past 2^31: one page over and
    over, then the page that holds the tree."""
    page, max_pages, N, D = 115264, 18631, 4, 64
    cap = page * max_pages
    assert 2 ** 31 - 128 < cap < 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(8)
    kp = torch.empty(2, page, 1, D, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    vp = torch.ones_like(kp)
    q = torch.empty(1, N, 2, D, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    table = torch.zeros(1, max_pages, dtype=torch.int32, device="cuda")
    table[0, -1] = 1
    parents = [-1, 0, 0, 2]
    see = torch.from_numpy(tp.tree_sees(parents, N)[0]).cuda()
    flat, rows = kp.reshape(-1, D).double(), q.reshape(-1, D).double()
    s = (rows @ flat.T * 0.125).reshape(N, 2, 2, page)  # node, head, page, row
    E = 68 * tp.U32 * 0.125 * float((rows.abs() @ flat.abs().T).max())
    body = torch.logsumexp(s[:, :, 0], -1) + np.log(max_pages - 1)
    for L in (cap - 9, cap):
        last = page - (cap - L)  # rows in use of the last page
        out, lse = fa.decode_tree(q, kp, vp, table, torch.tensor([L], dtype=torch.int32, device="cuda"),
                                  torch.tensor([parents], dtype=torch.int32, device="cuda"), 0.125,
                                  lse=True)
        torch.cuda.synchronize()
        assert fa.fa_device_error()[0] == fa.FA_OK
        tail = s[:, :, 1, :last].clone()
        tail[:, :, last - N:][~see[:, None].expand(N, 2, N)] = -torch.inf
        ref = torch.logaddexp(body, torch.logsumexp(tail, -1))
        # fp32 sums of a share's 2^31 / 128 / 152 tiles one after another, each
        # addition off by at most half a step; the scores' part as in check_tree.
        adds = cap / 128 / 152 + 200
        assert ((lse[0].double() - ref).abs() <= adds * tp.U32 + E + 2.0 ** -18).all()
        # O = 1 but for its sums: eight additions per tile, which may truncate.
        assert ((out.float() - 1).abs() <= 8 * adds * 2 * tp.U32 + adds * tp.U32 + 2.0 ** -7).all()


@pytest.mark.parametrize("T,Hq,Hkv,D", [(135000, 128, 8, 128), (8500001, 4, 2, 64)])
def test_weight_gradient_past_2_31_elements(fa, T, Hq, Hkv, D):
    """Single tokens on both sides of 2^31 elements, each counted once."""
    assert T * Hq * D > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(5)
    qkv = torch.empty(T, Hq + Hkv, D, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    q, k = qkv[:, :Hq], qkv[:, Hq:]
    w = torch.empty(D, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    f = (10000.0 ** (-torch.arange(D // 2, dtype=torch.float64) / (D // 2))).float()
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    edge = 2 ** 31 // (Hq * D)
    at = [0, 77777, edge - 1, edge, T - 1]
    go = [torch.zeros(T, H, D, dtype=torch.bfloat16, device="cuda") for H in (Hq, Hkv)]
    for x in go:
        x[at] = torch.empty(5, *x.shape[1:], device="cuda").normal_(generator=g).bfloat16()
    dq, dk, dqw, dkw = fa.qk_norm_rope_backward(*go, q, k, w, w, f.cuda(), pos, 1e-6)
    torch.cuda.synchronize()
    assert fa.fa_device_error()[0] == fa.FA_OK
    ang = tp.angles(at, f)
    for x, gr, dx, dw in ((q, go[0], dq, dqw), (k, go[1], dk, dkw)):
        tp.check_weight_grad(dw, x[at], w, gr[at], ang, 1e-6, False, 5 * x.shape[1])
        dx[at] = 0
        assert not dx.any()
