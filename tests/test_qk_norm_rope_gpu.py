"""Norm of queries and keys with rotary positions (fa_qk_norm_rope), its form
that writes cache pages and its gradient, against plain 64-bit forms, and the
gradient against differences."""
import random

import numpy as np
import pytest
import torch

from tests import tree_plain as tp

pytestmark = pytest.mark.gpu
EPS = 1e-5


def weights(D, dtype, g):
    return [(1 + 0.3 * torch.randn(D, generator=g)).to(dtype) for _ in range(2)]


def freqs(rot, theta=10000.0):
    i = torch.arange(rot // 2, dtype=torch.float64)
    return (theta ** (-2 * i / rot)).float()


def heads(T, Hq, Hkv, D, dtype, g, packed):
    if packed:
        x = torch.randn(T, Hq + 2 * Hkv + 1, D, generator=g).to(dtype).cuda()
        return x[:, :Hq], x[:, Hq:Hq + Hkv]
    return (torch.randn(T, Hq, D, generator=g).to(dtype).cuda(),
            torch.randn(T, Hkv, D, generator=g).to(dtype).cuda())


SHAPES = [
    # T, Hq, Hkv, D, rot, dtype, interleaved, packed
    (1, 1, 1, 64, 64, torch.bfloat16, False, False),
    (1, 128, 8, 128, 128, torch.bfloat16, False, True),
    (3, 5, 1, 128, 64, torch.float16, True, False),
    (130, 8, 2, 128, 128, torch.bfloat16, False, True),
    (257, 7, 7, 64, 16, torch.float16, False, True),
    (513, 3, 1, 64, 48, torch.bfloat16, True, True),
    (64, 9, 3, 128, 112, torch.float16, False, False),
    (5000, 2, 1, 128, 128, torch.bfloat16, True, False),
    # Several tokens per step: more tokens than resident warps, few heads.
    (9001, 4, 2, 64, 16, torch.float16, False, False),
    (7003, 8, 3, 64, 64, torch.bfloat16, True, True),
    (6001, 16, 1, 64, 48, torch.float16, False, True),
    (5999, 1, 1, 64, 64, torch.bfloat16, False, True),
    (4003, 8, 2, 128, 112, torch.bfloat16, False, True),
    (5003, 5, 3, 128, 64, torch.float16, True, False),
    (20011, 0, 2, 64, 32, torch.bfloat16, False, False),
]


@pytest.mark.parametrize("T,Hq,Hkv,D,rot,dtype,il,packed", SHAPES)
def test_forward(fa, T, Hq, Hkv, D, rot, dtype, il, packed):
    g = torch.Generator().manual_seed(T + D)
    q, k = heads(T, Hq, Hkv, D, dtype, g, packed)
    qw, kw = weights(D, dtype, g)
    pos = torch.randint(0, 100000, (T,), generator=g).int()
    f = freqs(rot)
    qo, ko = fa.qk_norm_rope(q, k, qw.cuda(), kw.cuda(), f.cuda(), pos.cuda(), EPS, interleaved=il)
    ang = tp.angles(pos.numpy(), f)
    tp.check_rope(qo, q, qw, ang, EPS, il)
    tp.check_rope(ko, k, kw, ang, EPS, il)


@pytest.mark.parametrize("T,Hq,Hkv,D,rot,dtype,il,packed", SHAPES)
def test_backward(fa, T, Hq, Hkv, D, rot, dtype, il, packed):
    g = torch.Generator().manual_seed(T + D + 1)
    q, k = heads(T, Hq, Hkv, D, dtype, g, packed)
    qw, kw = weights(D, dtype, g)
    pos = torch.randint(0, 5000, (T,), generator=g).int()
    f = freqs(rot)
    go = [torch.randn(T, H, D, generator=g).to(dtype).cuda() for H in (Hq, Hkv)]
    args = (q, k, qw.cuda(), kw.cuda(), f.cuda(), pos.cuda(), EPS)
    got = fa.qk_norm_rope_backward(*go, *args, interleaved=il)
    again = fa.qk_norm_rope_backward(*go, *args, interleaved=il)
    for a, b in zip(got, again):
        assert torch.equal(a, b)
    ang = tp.angles(pos.numpy(), f)
    h = tp.HALF[dtype]
    for x, w, gr, dx, dw in ((q, qw, go[0], got[0], got[2]), (k, kw, go[1], got[1], got[3])):
        rx, rw, sx, sw = tp.norm_rope_grad(x, w, gr, ang, EPS, il)
        # dx: one rounding, and at most 96 fp32 roundings of its two terms (the
        # dot product 24, the reciprocal root 14 in each of three powers, the
        # turn 11, 6 products and differences).
        tol = h * np.abs(rx) + (1 + h) * 96 * tp.U32 * sx + tp.TINY[dtype]
        assert np.all(np.abs(tp.f64(dx) - rx) <= tol)
        # dw: 40 roundings of each product, and the additions of a lane (at
        # most T H / 8 of them here), a block and the blocks.
        n = 40 + 13 + 40 + T * x.shape[1] // 8
        assert np.all(np.abs(tp.f64(dw) - rw) <= n * tp.U32 * sw)


def test_gradient_against_differences(fa):
    """Central differences of the 64-bit forward, along random directions.  The
    outputs are linear in the weights and smooth in x: with a step of 1e-6 the
    difference's own error is below 1e-8 of the sizes; the rest is the rounding
    of dq (a half step per element)."""
    T, Hq, Hkv, D, rot = 6, 2, 1, 64, 32
    g = torch.Generator().manual_seed(3)
    q, k = heads(T, Hq, Hkv, D, torch.bfloat16, g, False)
    qw, kw = weights(D, torch.bfloat16, g)
    pos = torch.arange(T).int()
    f = freqs(rot)
    go = [torch.randn(T, H, D, generator=g).bfloat16().cuda() for H in (Hq, Hkv)]
    dq, dk, dqw, dkw = fa.qk_norm_rope_backward(*go, q, k, qw.cuda(), kw.cuda(), f.cuda(),
                                                pos.cuda(), EPS)
    ang = tp.angles(pos.numpy(), f)
    rng = np.random.RandomState(0)
    for x, w, gr, dx, dw in ((q, qw, go[0], dq, dqw), (k, kw, go[1], dk, dkw)):
        def loss(xx, ww):
            y = xx / np.sqrt((xx * xx).mean(-1, keepdims=True) + EPS) * ww
            return float((tp.turn(y, ang, False) * tp.f64(gr)).sum())
        x0, w0 = tp.f64(x), tp.f64(w)
        for _ in range(4):
            u, t = rng.randn(*x0.shape), rng.randn(D)
            e = 1e-6
            num = (loss(x0 + e * u, w0) - loss(x0 - e * u, w0)) / (2 * e)
            ours = float((tp.f64(dx) * u).sum())
            assert abs(num - ours) <= 2.0 ** -8 * float((np.abs(tp.f64(dx) * u)).sum()) + 1e-4
            num = (loss(x0, w0 + e * t) - loss(x0, w0 - e * t)) / (2 * e)
            assert abs(num - float((tp.f64(dw) * t).sum())) <= 1e-3


def test_far_and_negative_positions(fa):
    """fp32 products of position and frequency would be whole turns off."""
    pos = torch.tensor([0, 1, -1, 1 << 20, (1 << 24) + 1, 2 ** 31 - 1, -2 ** 31, 123456789],
                       dtype=torch.int32)
    g = torch.Generator().manual_seed(9)
    q, k = heads(len(pos), 4, 2, 128, torch.float16, g, False)
    qw, kw = weights(128, torch.float16, g)
    f = freqs(128, 1e6)
    qo, ko = fa.qk_norm_rope(q, k, qw.cuda(), kw.cuda(), f.cuda(), pos.cuda(), EPS)
    # The fractions are off by at most 2^-54 of a turn (products of 53 bits of
    # numbers below 1/4): 2 pi 2^-23 at 2^31, 13 fp32 roundings of the pair.
    ang = tp.angles(pos.numpy(), f)
    for got, x, w in ((qo, q, qw), (ko, k, kw)):
        ref, size = tp.norm_rope(x, w, ang, EPS, False)
        tol = 2.0 ** -11 * np.abs(ref) + 46 * tp.U32 * size + 2.0 ** -25
        assert np.all(np.abs(tp.f64(got) - ref) <= tol)


def test_in_place_and_strides(fa):
    g = torch.Generator().manual_seed(4)
    q, k = heads(70, 6, 2, 128, torch.bfloat16, g, False)
    qw, kw = (w.cuda() for w in weights(128, torch.bfloat16, g))
    pos = torch.arange(70, dtype=torch.int32, device="cuda")
    f = freqs(128).cuda()
    qo, ko = fa.qk_norm_rope(q, k, qw, kw, f, pos, EPS)
    q5 = q.reshape(2, 5, 7, 6, 128)
    q2, k2 = fa.qk_norm_rope(q5, k.reshape(2, 5, 7, 2, 128), qw, kw, f, pos.reshape(2, 5, 7), EPS)
    assert torch.equal(q2.reshape(qo.shape), qo) and torch.equal(k2.reshape(ko.shape), ko)
    fa.qk_norm_rope(q, k, qw, kw, f, pos, EPS, q_out=q, k_out=k)
    assert torch.equal(q, qo) and torch.equal(k, ko)
    go = [torch.randn(70, H, 128, generator=g).bfloat16().cuda() for H in (6, 2)]
    a = fa.qk_norm_rope_backward(*go, qo, ko, qw, kw, f, pos, EPS)
    st = fa.fa_qk_norm_rope_backward(go[0].data_ptr(), go[1].data_ptr(), qo.data_ptr(),
                                     ko.data_ptr(), qw.data_ptr(), kw.data_ptr(), f.data_ptr(),
                                     pos.data_ptr(), go[0].data_ptr(), go[1].data_ptr(),
                                     a[2].data_ptr(), a[3].data_ptr(), 70, 6, 2, 128, 128, 768, 256,
                                     EPS, 0, fa.FA_BF16, torch.cuda.current_stream().cuda_stream)
    assert st == fa.FA_OK and torch.equal(go[0], a[0]) and torch.equal(go[1], a[1])


def test_no_tokens(fa):
    q, k = torch.empty(0, 4, 64, dtype=torch.float16).cuda(), torch.empty(0, 2, 64, dtype=torch.float16).cuda()
    w = torch.ones(64, dtype=torch.float16).cuda()
    f, pos = freqs(64).cuda(), torch.empty(0, dtype=torch.int32).cuda()
    assert fa.qk_norm_rope(q, k, w, w, f, pos, EPS)[0].shape == q.shape
    grads = fa.qk_norm_rope_backward(q, k, q, k, w, w, f, pos, EPS)
    assert not grads[2].any() and not grads[3].any()


@pytest.mark.parametrize("B,N,Hq,Hkv,D,page,lens,dtype,il,own_pos", [
    (1, 1, 8, 2, 128, 64, [1], torch.bfloat16, False, False),
    (4, 5, 6, 3, 64, 32, [5, 0, 100, 4], torch.float16, True, True),
    (3, 64, 16, 1, 128, 96, [64, 300, 97], torch.bfloat16, False, True),
    (20, 2, 4, 4, 64, 32, [2 + 31 * i for i in range(20)], torch.bfloat16, False, False),
    # Several tokens per step, some of one sequence and some of the next.
    (71, 43, 6, 3, 64, 32, [43 + 5 * i if i % 7 else i for i in range(71)], torch.float16, True, False),
    (70, 37, 8, 1, 128, 64, [37 + 3 * i if i % 9 else 0 for i in range(70)], torch.bfloat16, False, True),
])
def test_append(fa, B, N, Hq, Hkv, D, page, lens, dtype, il, own_pos):
    g = torch.Generator().manual_seed(B + N)
    rng = random.Random(B)
    max_pages = max(1, -(-max(lens) // page))
    P = B * max_pages + 2
    kp0 = torch.randn(P, page, Hkv, D, generator=g).to(dtype)
    vp0 = torch.randn(P, page, Hkv, D, generator=g).to(dtype)
    table = torch.randperm(P, generator=g)[:B * max_pages].reshape(B, max_pages).int()
    qkv = torch.randn(B, N, Hq + 2 * Hkv, D, generator=g).to(dtype).cuda()
    q, k, v = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:]
    qw, kw = weights(D, dtype, g)
    f = freqs(D)
    slots = np.array(lens)[:, None] - N + np.arange(N)
    pos = torch.tensor([[rng.randint(0, 9999) for _ in range(N)] for _ in range(B)]).int() if own_pos else None
    kp, vp = kp0.cuda(), vp0.cuda()
    qo = fa.qk_norm_rope_append(q, k, v, qw.cuda(), kw.cuda(), f.cuda(), kp, vp, table.cuda(),
                                torch.tensor(lens, dtype=torch.int32).cuda(), EPS,
                                positions=None if pos is None else pos.cuda(), interleaved=il)
    torch.cuda.synchronize()
    assert fa.fa_device_error()[0] == fa.FA_OK
    ang = tp.angles(slots if pos is None else pos.numpy(), f)
    tp.check_rope(qo, q, qw, ang, EPS, il)
    kp, vp = kp.cpu(), vp.cpu()
    for b, L in enumerate(lens):
        if L < N:
            continue
        for s in range(N):
            t = int(slots[b, s])
            pid = int(table[b, t // page])
            tp.check_rope(kp[pid, t % page][None], k[b, s][None].cpu(), kw, ang[b, s][None], EPS, il)
            assert torch.equal(vp[pid, t % page], v[b, s].cpu())
            kp[pid, t % page], vp[pid, t % page] = kp0[pid, t % page], vp0[pid, t % page]
    assert torch.equal(kp, kp0) and torch.equal(vp, vp0)  # nothing else was written


@pytest.mark.parametrize("H,T", [(4, 9000), (16, 30000)])
def test_rows_at_the_ends_of_their_memory(fa, H, T):
    """Loads of several tokens per step stay in the rows: q is the end of a tensor
    whose other rows are NaN, and the outputs are the same as alone."""
    g = torch.Generator().manual_seed(T)
    q, k = heads(T, H, 1, 64, torch.bfloat16, g, False)
    qw, kw = (w.cuda() for w in weights(64, torch.bfloat16, g))
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    f = freqs(64).cuda()
    ref = fa.qk_norm_rope(q, k, qw, kw, f, pos, EPS)
    big = torch.full((T + 7, H + 3, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    big[7:, 3:] = q
    got = fa.qk_norm_rope(big[7:, 3:], k, qw, kw, f, pos, EPS)
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])


def test_append_with_bad_pages_and_lengths(fa):
    B, N, D = 3, 4, 64
    g = torch.Generator().manual_seed(1)
    kp0 = torch.randn(8, 32, 1, D, generator=g).bfloat16()
    table = torch.tensor([[0, 99], [1, 2], [3, 4]], dtype=torch.int32)
    lens = torch.tensor([34, 65, 30], dtype=torch.int32)  # half on a bad page; past the table; sound
    qkv = torch.randn(B, N, 3, D, generator=g).bfloat16().cuda()
    w = torch.ones(D).bfloat16().cuda()
    kp, vp = kp0.cuda(), kp0.cuda()
    fa.qk_norm_rope_append(qkv[:, :, :1], qkv[:, :, 1:2], qkv[:, :, 2:], w, w, freqs(D).cuda(), kp, vp,
                           table.cuda(), lens.cuda(), EPS)
    st, _ = fa.fa_device_error()
    assert st == fa.FA_ERR_BOUNDS
    want = kp0.clone()
    want[0, 30], want[0, 31] = qkv[0, 0, 2:].cpu(), qkv[0, 1, 2:].cpu()
    for s in range(N):
        want[3, 26 + s] = qkv[2, s, 2:].cpu()
    assert torch.equal(vp.cpu(), want)
    assert fa.fa_device_error()[0] == fa.FA_OK


@pytest.mark.parametrize("T,Hq,Hkv,D,rot,dtype,il,packed", SHAPES + [
    (2432, 16, 16, 128, 128, torch.bfloat16, False, True),
    (4865, 16, 5, 128, 128, torch.float16, True, False),
    (3001, 33, 31, 64, 64, torch.bfloat16, False, False),
])
def test_weight_gradient_to_its_own_additions(fa, T, Hq, Hkv, D, rot, dtype, il, packed):
    """Within the additions that a lane really makes, which no lost or doubled
    group of rows can hide in (test_weight_grad_check.py plants some)."""
    g = torch.Generator().manual_seed(T + D + 2)
    q, k = heads(T, Hq, Hkv, D, dtype, g, packed)
    qw, kw = weights(D, dtype, g)
    pos = torch.randint(0, 5000, (T,), generator=g).int()
    f = freqs(rot)
    go = [torch.randn(T, H, D, generator=g).to(dtype).cuda() for H in (Hq, Hkv)]
    got = fa.qk_norm_rope_backward(*go, q, k, qw.cuda(), kw.cuda(), f.cuda(), pos.cuda(), EPS,
                                   interleaved=il)
    adds = tp.lane_additions(T, Hq, Hkv, D, torch.cuda.get_device_properties(0).multi_processor_count)
    ang = tp.angles(pos.numpy(), f)
    tp.check_weight_grad(got[2], q, qw, go[0], ang, EPS, il, adds)
    tp.check_weight_grad(got[3], k, kw, go[1], ang, EPS, il, adds)


@pytest.mark.parametrize("T,Hq,Hkv,D,rot,dtype,il,packed", [s for s in SHAPES if s[0] > 100])
def test_single_tokens_reach_the_weight_gradient(fa, T, Hq, Hkv, D, rot, dtype, il, packed):
    """A gradient of zero but for a few tokens, the first and the last among
    them: each counts once, and the other tokens' dx is zero."""
    g = torch.Generator().manual_seed(T + D + 3)
    q, k = heads(T, Hq, Hkv, D, dtype, g, packed)
    qw, kw = weights(D, dtype, g)
    pos = torch.randint(0, 5000, (T,), generator=g).int()
    f = freqs(rot)
    at = sorted({0, T - 1, *torch.randint(0, T, (4,), generator=g).tolist()})
    go = [torch.zeros(T, H, D, dtype=dtype).cuda() for H in (Hq, Hkv)]
    for x in go:
        x[at] = torch.randn(len(at), *x.shape[1:], generator=g).to(dtype).cuda()
    got = fa.qk_norm_rope_backward(*go, q, k, qw.cuda(), kw.cuda(), f.cuda(), pos.cuda(), EPS,
                                   interleaved=il)
    ang = tp.angles(pos.numpy()[at], f)
    for x, w, gr, dx, dw in ((q, qw, go[0], got[0], got[2]), (k, kw, go[1], got[1], got[3])):
        tp.check_weight_grad(dw, x[at], w, gr[at], ang, EPS, il, len(at) * x.shape[1])
        dx[at] = 0
        assert not dx.any()
