"""Sampling (fa_sample): the search for top-p's border where the first estimate, counts in
bins times the weight of a bin's middle, misses it."""
import numpy as np
import pytest
import torch

from tests import serving_plain as sp
from tests.test_sample_gpu import DT, check

pytestmark = pytest.mark.gpu


def bits(t):
    return t.view(torch.int32)


def below_the_first_list(V, rng):
    """A row, and a top_p, whose border lies below what the first list holds (temperature 1).
    Hundreds of tokens at the lower edges of their bins (1/64 wide), so that the estimate makes
    them too heavy; a few tokens, among which it finds the border; then, a gap below, tokens at
    the upper edges of theirs, among whose first ones the border is."""
    x = -60.0 + rng.normal(0, 1, V)
    n1, n2, n3 = int(rng.integers(300, 900)), int(rng.integers(10, 60)), int(rng.integers(400, 1500))
    at = rng.permutation(V)[:n1 + n2 + n3]
    x[at[0]] = 0.0
    x[at[1:n1]] = -(2.5 + (rng.integers(0, 32, n1 - 1) + 0.45) / 64)
    x[at[n1:n1 + n2]] = -(3.2 + rng.uniform(0, 0.8, n2))
    x[at[n1 + n2:]] = -(4.5 + (rng.integers(0, 32, n3) - 0.45) / 64)
    x = x.astype(np.float32)
    w = np.exp(x.astype(np.float64))
    return x, float(w[x > -4.2].sum() / w.sum() + rng.uniform(-0.0005, 0.0015))


# Rows and vocabularies of clusters of 1, 2, 4 and 8 CTAs.
@pytest.mark.parametrize("dtype", ["fp32", "fp16"])
@pytest.mark.parametrize("R,V", [(300, 6000), (200, 8000), (64, 8000), (40, 33000)])
def test_border_below_the_first_list(fa, R, V, dtype):
    """List after list, beside rows that are done sooner: the tokens and distributions of the
    64-bit form, and the same bits every time."""
    rng = np.random.default_rng(V + R)
    rows = [below_the_first_list(V, rng) for _ in range(R)]
    x = torch.from_numpy(np.stack([r[0] for r in rows])).to(DT[dtype])
    p = [tp if r % 4 else 1.0 for r, (_, tp) in enumerate(rows)]
    k = [0 if r % 8 else 20 for r in range(R)]
    u = rng.random(R).astype(np.float32).tolist()
    t0, p0 = check(fa, x, u, k=k, p=p)
    f = lambda v, t: torch.tensor(v, dtype=t, device="cuda")  # noqa: E731
    xd, args = x.cuda(), dict(top_k=f(k, torch.int32), top_p=f(p, torch.float32), probs=True)
    for _ in range(100):
        t1, p1 = fa.sample(xd, f(u, torch.float32), **args)
        assert torch.equal(t0, t1) and torch.equal(bits(p0), bits(p1))


def equal_bins(n):
    """Twelve tokens in the middle of each of the estimate's bins from 2 temperatures down, a
    largest one; and the shares of the weight that end with a bin of the next thread's."""
    x = np.concatenate([[0.0], -np.repeat((np.arange(513, 1100) - 385) / 64, 12)]).astype(np.float32)
    w = np.exp(x.astype(np.float64))
    ends = np.cumsum(w)[[12 * (4 * t - 513) for t in range(130, 130 + n)]] / w.sum()
    return x, ends


@pytest.mark.parametrize("dtype", ["fp32", "fp16"])
def test_top_p_on_the_estimates_borders(fa, dtype):
    """Consecutive values of top_p around sums that end with a thread's bins: there, by the
    rounding of its sums, more than one thread or none finds the border's bin."""
    rng = np.random.default_rng(3)
    x, ends = equal_bins(8)
    p = [float(np.float32(e) + np.float32(k * 2.0 ** -24)) for e in ends for k in range(-12, 13)]
    order = rng.permutation(len(x))
    x = torch.from_numpy(x[order])[None].expand(len(p), -1).contiguous().to(DT[dtype])
    u = rng.random(len(p)).astype(np.float32).tolist()
    t0, p0 = check(fa, x, u, p=p)
    f = lambda v: torch.tensor(v, device="cuda")  # noqa: E731
    xd = x.cuda()
    for at in (slice(None), slice(0, 60)):  # clusters of 2 and of 4
        for _ in range(40):
            t1, p1 = fa.sample(xd[at], f(u)[at], top_p=f(p)[at], probs=True)
            assert torch.equal(t0[at], t1) and torch.equal(bits(p0[at]), bits(p1))


def time_of(fa, x, u, **settings):
    """Microseconds of a call."""
    def run(n):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        for _ in range(n):
            fa.sample(x, u, **settings)
        b.record()
        b.synchronize()
        return a.elapsed_time(b) * 1e3 / n
    run(3)
    return min(run(5) for _ in range(3))


def settings_of(R, T, p):
    return dict(temperature=torch.full((R,), T, device="cuda"), top_p=torch.full((R,), p, device="cuda"))


@pytest.mark.parametrize("V,T,scale,p", [
    (5000, 1e-7, 2.5, 0.9),          # differences of logits are millions of temperatures
    (1431, 4930.0, 2.0 ** 60, 0.5),  # the same, far from 0
    (5000, 2.0 ** -99, 2.5, 0.95),   # the lowest temperature that counts
    (5000, 1.0, 2.0 ** -21, 1 - 2.0 ** -20),  # nearly equal logits of which nearly all stay
])
def test_no_row_is_looked_for_long(fa, V, T, scale, p):
    """Rows whose border the bins do not show are found by halving: a call takes some tens of
    rounds, not thousands (42 rounds of less than a plain call each; 20000 would be hundreds)."""
    g = torch.Generator().manual_seed(V)
    x = torch.randn(8, V, generator=g) * scale
    if scale < 1:
        x = 5.0 + torch.rand(8, V, generator=g) * 2 * scale - scale
    u = torch.rand(8, generator=g).tolist()
    check(fa, x, u, T=[T] * 8, p=[p] * 8)
    xd, ud = x.cuda(), torch.tensor(u, device="cuda")
    plain = torch.randn(8, V, generator=g).cuda()
    assert time_of(fa, xd, ud, **settings_of(8, T, p)) < 42 * time_of(fa, plain, ud, **settings_of(8, 1.0, 0.9))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("T,at,scale", [(1e-7, 0.0, 2.5), (0.01, 1e5, 2.0), (0.3, -3e4, 2.0), (4930.0, 0.0, 2.0 ** 60),
                                        (2.0 ** -99, 0.0, 2.5), (1e-4, 20.0, 3.0)])
def test_many_temperatures_from_zero(fa, T, at, scale, dtype):
    """The estimate holds however many temperatures the logits are from 0: a call takes what one
    near 0 does (three times is allowed; without it the search halves, six times and more)."""
    g = torch.Generator().manual_seed(21)
    x = (at + torch.randn(8, 5000, generator=g) * scale).to(DT[dtype])
    u = torch.rand(8, generator=g).tolist()
    p = [0.9013, 0.3007, 0.9991, 0.5511, 0.7023, 0.9517, 0.1111, 0.4303]
    check(fa, x, u, T=[T] * 8, p=p)
    check(fa, x, u, T=[T] * 8, p=p, m=[0.01] * 8, k=[0, 4000] * 4)
    if dtype == "fp32":
        xd, ud = x.cuda(), torch.tensor(u, device="cuda")
        plain = torch.randn(8, 5000, generator=g).cuda()
        assert time_of(fa, xd, ud, **settings_of(8, T, 0.9)) < 3 * time_of(fa, plain, ud, **settings_of(8, 1.0, 0.9))


@pytest.mark.parametrize("seed", [0, 1, 2])
def test_target_within_the_sums_rounding_of_a_border(fa, seed):
    """Half a million rows whose top_p is the float next to the share of their first tokens:
    some targets lie within the rounding of the sums, which one round may put above a border
    and the next below it.  Either answer is one token off at most; none keeps everything.
    (Tokens at bins' edges, so that the first look is below the border and a second follows.)"""
    R, n1, n3 = 1 << 19, 200, 100
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda n: torch.randint(0, 32, (R, n), device="cuda", generator=g).float()  # noqa: E731
    x = torch.cat([torch.zeros(R, 1, device="cuda"), -(2.5 + (r(n1 - 1) - 0.45) / 64),
                   -(4.2 + (r(n3) + 0.45) / 64)], dim=1)
    w = x.double().exp()
    p = (w[:, :n1].sum(1) / w.sum(1)).float()
    perm = torch.randperm(x.shape[1], device="cuda", generator=g)
    x, w = x[:, perm].contiguous(), w[:, perm]
    _, probs = fa.sample(x, torch.rand(R, device="cuda", generator=g), top_p=p, probs=True)
    kept = (w * (probs > 0)).sum(1) / w.sum(1)
    # One of the second kind more is at most e^-4.2 / (1 + 199 e^-3) < 0.0014 of the weight, one of
    # the first missing e^-2.49 / (1 + 199 e^-3) < 0.0077.
    assert int((kept > p + 0.0014).sum()) == 0 and int((kept < p - 0.0077).sum()) == 0


@pytest.mark.parametrize("T", [2.0 ** -149, 2.0 ** -148, 2.0 ** -130, 2.0 ** -120, 2.0 ** -100, 2.0 ** -99])
def test_temperatures_below_the_least(fa, T):
    """They count as 2^-99: in the weights, in min-p's border, and in how far top-p's search
    steps.  Logits of a few such temperatures, and ordinary ones."""
    g = torch.Generator().manual_seed(31)
    x = torch.randn(12, 3000, generator=g) * 2
    x[:8] *= 2.0 ** -100
    x[0] = -1.0
    x[0, 100], x[0, 2000] = 0.0, -(2.0 ** -100)   # weights 1 and e^-1/2
    u = torch.rand(12, generator=g).tolist()
    u[0] = 0.8
    k, p, m = [0, 40, 0] * 4, [1.0, 1.0, 0.9, 0.5] * 3, [0.5, 0.0, 0.3, 0.0, 0.0, 0.2] * 2
    f = lambda v, t=torch.float32: torch.tensor(v, dtype=t, device="cuda")  # noqa: E731
    tokens, probs = fa.sample(x.cuda(), f(u), temperature=f([T] * 12), top_k=f(k, torch.int32), top_p=f(p),
                              min_p=f(m), probs=True)
    f32 = lambda v: float(np.float32(v))  # noqa: E731
    for r in range(12):
        tok, dist, margin = sp.sample(x[r].double().numpy(), f32(u[r]), 2.0 ** -99, k[r], f32(p[r]), f32(m[r]))
        assert margin > 1e-9 and int(tokens[r]) == tok, r
        assert np.array_equal(probs[r].cpu().numpy() > 0, dist > 2.0 ** -119), r
    assert int(tokens[0]) == 2000 and int((probs[0] > 0).sum()) == 2


@pytest.mark.parametrize("dtype,unit", [("fp32", 2.0 ** -149), ("fp32", 2.0 ** -60), ("bf16", 2.0 ** -133),
                                        ("bf16", 2.0 ** -60), ("fp16", 2.0 ** -24), ("fp16", 2.0 ** -14)])
def test_bounds_of_the_search_around_zero(fa, dtype, unit):
    """Logits of a few units to either side of 0, many of them 0: the search's bounds come to lie
    between 0 and the largest negative number, and 0 is on one side of them."""
    g = torch.Generator().manual_seed(41)
    R, V = 48, 4999
    x = (torch.randint(-40, 41, (R, V), generator=g).double() * unit).to(DT[dtype])
    x[::2, ::3] = 0.0
    x[1::4, ::5] = -0.0
    u = torch.rand(R, generator=g).tolist()
    p = [(r + 0.5371) / R for r in range(R)]
    check(fa, x, u, p=p)
    check(fa, x, u, T=[0.01 + 0.1 * r for r in range(R)], p=p, m=[0.0, 0.5] * (R // 2))
    check(fa, x, u, p=p, k=[100 * r for r in range(R)])
    check(fa, x, u, k=[100 * r + 1 for r in range(R)])


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
def test_min_p_that_ends_at_zero(fa, dtype):
    """Of logits up to 0, the zeros alone with min_p = 1; of logits up to 1, those from 0 on with
    the number before 1 / e (16-bit logits; T ln(min_p) + 1 is just below 0)."""
    g = torch.Generator().manual_seed(42)
    x = -torch.rand(12, 3001, generator=g) - 2.0 ** -10
    x[:, 5:40:7] = 0.0
    x[::3, 2000:2100] = -0.0
    u = torch.rand(12, generator=g).tolist()
    p = [0.1 + 0.0713 * r for r in range(12)]
    check(fa, x.to(DT[dtype]), u, p=p, m=[1.0] * 12)
    check(fa, x.to(DT[dtype]), u, p=p, m=[1.0] * 12, T=[0.2 + r for r in range(12)])
    if dtype != "fp32":
        x[:, 77] = 1.0
        below = float(np.nextafter(np.float32(np.exp(-1.0)), np.float32(0)))
        check(fa, x.to(DT[dtype]), u, p=[0.999 - 0.001 * r for r in range(12)], m=[below] * 12)


@pytest.mark.parametrize("m", [1.0000001, 3.0, float("inf")])
def test_min_p_above_1_keeps_one_token(fa, m):
    """No weight reaches it, and one token is kept at least: the lowest of the largest, of which
    there are several."""
    g = torch.Generator().manual_seed(43)
    x = torch.randn(6, 2003, generator=g).clamp(max=1.5)
    u = torch.rand(6, generator=g).tolist()
    for kw in (dict(), dict(p=[0.9] * 6), dict(k=[50] * 6), dict(k=[700] * 6, p=[0.5] * 6), dict(T=[0.0] * 6)):
        tokens, probs = check(fa, x, u, m=[m] * 6, **kw)
        assert ((probs > 0).sum(-1) == 1).all()
