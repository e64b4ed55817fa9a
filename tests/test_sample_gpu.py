"""Sampling (fa_sample) against a plain 64-bit form: the tokens are whole numbers and
have to be equal; a case whose u or top_p lies within 1e-9 of a border in the plain form
is not looked at (the inputs are such that there is none, which is checked)."""
import numpy as np
import pytest
import torch

from tests import serving_plain as sp

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def check(fa, logits, u, T=None, k=None, p=None, m=None, probs=True, status=None):
    """logits [R, V] on the CPU (or a CUDA view), settings lists or None."""
    dev = "cuda"
    x = logits.to(dev) if not logits.is_cuda else logits
    f = lambda v, t: None if v is None else torch.tensor(v, dtype=t, device=dev)  # noqa: E731
    out = fa.sample(x, f(u, torch.float32), temperature=f(T, torch.float32), top_k=f(k, torch.int32),
                    top_p=f(p, torch.float32), min_p=f(m, torch.float32), probs=probs)
    torch.cuda.synchronize()
    st, detail = fa.fa_device_error()
    assert st == fa.FA_OK, hex(detail)
    tokens, pr = out if probs else (out, None)
    f32 = lambda v: float(np.float32(v))  # noqa: E731
    rows = x.float().cpu().double().numpy()
    for r in range(rows.shape[0]):
        tok, dist, margin = sp.sample(rows[r], f32(u[r]), 1.0 if T is None else f32(T[r]),
                                      0 if k is None else k[r], 1.0 if p is None else f32(p[r]),
                                      0.0 if m is None else f32(m[r]))
        assert margin > 1e-9, (r, margin)
        assert int(tokens[r]) == tok, r
        if pr is not None:
            # Weights to 2^-31 (a hundredth of a rounding to fp32 is 2^-30.6), their sum and
            # quotient in pairs, one rounding to fp32; what is below fp32's normal range by
            # its half step.
            got = pr[r].double().cpu().numpy()
            err = np.abs(got - dist)
            assert np.all(err <= 2.0 ** -24 * dist * 1.01 + 2.0 ** -120), (r, err.max())
            assert np.array_equal(got > 0, dist > 2.0 ** -119) or np.all(dist[(got > 0) != (dist > 0)] < 1e-30)
    return tokens, pr


def rows_of(R, V, dtype, seed, sharp=2.5):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(R, V, generator=g) * sharp).to(DT[dtype]), torch.rand(R, generator=g).tolist(), g


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("R,V", [(1, 1), (2, 2), (3, 17), (5, 127), (4, 128), (6, 1000), (3, 4097), (7, 32000),
                                 (2, 50257), (3, 128256), (1, 262144)])
def test_temperature_alone(fa, R, V, dtype):
    x, u, g = rows_of(R, V, dtype, seed=V)
    T = [0.3 + 0.4 * i for i in range(R)]
    check(fa, x, u, T=T)


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("R,V,seed", [(8, 50, 0), (6, 999, 1), (12, 5003, 2), (9, 32000, 3), (4, 129280, 4)])
def test_all_filters(fa, R, V, seed, dtype):
    """Each row with settings of its own: filters on and off, k of 1, few, many, all but one."""
    x, u, g = rows_of(R, V, dtype, seed)
    pick = lambda v: [v[int(torch.randint(len(v), (1,), generator=g))] for _ in range(R)]  # noqa: E731
    T = pick([0.0, 0.2, 0.7, 1.0, 1.7])
    k = pick([0, 1, 2, 40, 333, V - 1, V, V + 9, -3])
    p = pick([1.0, 0.95, 0.9, 0.5, 0.999, 0.05, 1.5])
    m = pick([0.0, 0.001, 0.02, 0.3, -1.0])
    check(fa, x, u, T, k, p, m)
    check(fa, x, u, T, k=k, probs=False)
    check(fa, x, u, T, p=p)
    check(fa, x, u, m=m)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("V", [300, 20000])
def test_equal_logits(fa, V, dtype):
    """Ties: all equal, two values, few values; cuts inside them go by index."""
    g = torch.Generator().manual_seed(V)
    x = torch.zeros(5, V)
    x[1, ::3] = 1.0
    x[2] = torch.randint(0, 3, (V,), generator=g).float()
    x[3] = torch.randint(-1, 1, (V,), generator=g).float() * 0.0   # 0 and -0 are equal
    x[4] = -7.25
    x = x.to(DT[dtype])
    u = [0.4321, 0.777, 0.05, 0.9, 0.31]
    for k in (None, [5, 7, V // 2 + 1, V - 1, 3]):
        for p in (None, [0.37, 0.81, 0.93, 0.113, 0.555]):
            check(fa, x, u, k=k, p=p)
            check(fa, x, u, T=[0.0] * 5, k=k, p=p)


def test_infinities_nan_and_rows_without_any(fa):
    V = 700
    g = torch.Generator().manual_seed(1)
    x = torch.randn(8, V, generator=g)
    x[0, 5] = float("inf")
    x[1, ::50] = float("inf")
    x[2, ::2] = float("-inf")
    x[3] = float("-inf")
    x[4] = float("nan")
    x[5, 1::2] = float("nan")
    x[6] = float("-inf")
    x[6, 699] = -3e38
    x[7, 0] = 3e38
    u = [0.2, 0.61, 0.3, 0.5, 0.5, 0.7, 0.99, 0.4]
    for k in (None, [3] * 8, [699] * 8):
        for p in (None, [0.9] * 8):
            for m in (None, [0.1] * 8):
                tok, pr = check(fa, x, u, k=k, p=p, m=m)
                assert tok[3] == -1 and tok[4] == -1 and not pr[3:5].any()


def test_temperatures_at_the_ends(fa):
    x, u, _ = rows_of(8, 900, "fp32", 5)
    T = [1e-30, 1e-3, 1e30, float("inf"), 0.0, -1.0, float("nan"), 2.0 ** -126]
    check(fa, x, u, T)
    check(fa, x, u, T, p=[0.7] * 8)


def test_uniforms_at_the_ends(fa):
    """u = 0: the lowest kept token; 1 and above, which it should not be: the last; NaN as 0."""
    x, _, _ = rows_of(4, 600, "fp32", 6)
    tok, pr = fa.sample(x.cuda(), torch.tensor([0.0, 1.0, 7.0, float("nan")], device="cuda"),
                        top_k=torch.full((4,), 9, dtype=torch.int32, device="cuda"), probs=True)
    kept = [torch.nonzero(r)[:, 0].tolist() for r in pr.cpu()]
    assert all(len(r) == 9 for r in kept)
    assert tok.tolist() == [kept[0][0], kept[1][-1], kept[2][-1], kept[3][0]]


def test_borders_belong_to_the_token_above(fa):
    """Weights of 1/8 each: u on a border draws the token behind it; top_p on a border
    does not keep the token behind it."""
    x = torch.zeros(6, 8, device="cuda")
    u = torch.tensor([0.0, 0.125, 0.25 - 2.0 ** -26, 0.5, 0.875, 1 - 2.0 ** -24], device="cuda")
    assert fa.sample(x, u).tolist() == [0, 1, 1, 4, 7, 7]
    p = torch.tensor([0.125, 0.25, 0.2501, 0.5, 0.875, 2.0 ** -20], device="cuda")
    _, pr = fa.sample(x, u, top_p=p, probs=True)
    assert (pr > 0).sum(-1).tolist() == [1, 2, 3, 4, 7, 1]


@pytest.mark.parametrize("dtype", ["fp32", "fp16"])
def test_rows_of_a_larger_tensor(fa, dtype):
    """Strided rows that begin at every alignment, and what lies between them does not count."""
    V = 1001
    g = torch.Generator().manual_seed(9)
    big = (torch.randn(9, V + 13, generator=g) * 2).to(DT[dtype]).cuda()
    big[:, V + 5:] = 50.0
    big[:, :5] = 60.0
    u = torch.rand(9, generator=g).tolist()
    check(fa, big[:, 5:V + 5], u, p=[0.9] * 9)
    shaped = big[:8].reshape(2, 4, V + 13)[:, :, 5:V + 5]
    t, pr = fa.sample(shaped, torch.tensor(u[:8], device="cuda").reshape(2, 4), probs=True)
    assert t.shape == (2, 4) and pr.shape == shaped.shape
    assert t.flatten().tolist() == check(fa, big[:8, 5:V + 5], u[:8])[0].tolist()


def test_logits_that_stand_in_order(fa):
    """Rising and falling rows: all of the largest in one warp's part."""
    V = 40000
    up = torch.arange(V).float() * 1e-3
    x = torch.stack([up, up.flip(0), up.roll(V // 2)])
    for k in (None, [700, 5, 33]):
        for p in (None, [0.99, 0.5, 0.9]):
            check(fa, x, [0.123, 0.8, 0.5], k=k, p=p)


def test_drawn_as_often_as_the_distribution_says(fa):
    """20000 draws of one row: counts within 6 standard deviations."""
    R, V = 20000, 64
    g = torch.Generator(device="cuda").manual_seed(3)
    row = torch.randn(V, device="cuda", generator=g) * 2
    u = torch.rand(R, device="cuda", generator=g)
    tok, pr = fa.sample(row.expand(R, V).contiguous(), u, top_p=torch.full((R,), 0.9, device="cuda"),
                        probs=True)
    p = pr[0].double()
    n = torch.bincount(tok.long(), minlength=V).double()
    assert ((n - R * p).abs() <= 6 * (R * p * (1 - p)).sqrt() + 1e-9).all()


def test_equal_calls_give_equal_bits(fa):
    x, u, _ = rows_of(40, 33000, "fp32", 12)
    a = (x.cuda(), torch.tensor(u, device="cuda"))
    kw = dict(top_p=torch.full((40,), 0.93, device="cuda"), probs=True)
    t0, p0 = fa.sample(*a, **kw)
    for _ in range(5):
        t1, p1 = fa.sample(*a, **kw)
        assert torch.equal(t0, t1) and torch.equal(p0, p1)
