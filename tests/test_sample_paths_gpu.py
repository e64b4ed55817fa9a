"""Sampling (fa_sample) where its ways part: k around what a list holds, ties that overflow
it, borders near zero, rows of few finite logits, logits far from zero, weights that come
from a few or from all tokens, more rows than fit at once, the largest vocabularies."""
import pytest
import torch

from tests.test_sample_gpu import DT, check

pytestmark = pytest.mark.gpu


def gen(seed):
    return torch.Generator().manual_seed(seed)


def us(R, g):
    return torch.rand(R, generator=g).tolist()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("V", [513, 9000, 64000])
def test_k_around_the_lists_length(fa, V, dtype):
    g = gen(V)
    k = [31, 32, 33, 170, 171, 341, 342, 383, 384, 385, 512, 511]
    x = (torch.randn(len(k), V, generator=g) * 2).to(DT[dtype])
    u = us(len(k), g)
    check(fa, x, u, k=k)
    check(fa, x, u, T=[0.7] * len(k), k=k, p=[0.8] * len(k), m=[0.01] * len(k))


@pytest.mark.parametrize("dtype", ["fp32", "fp16"])
def test_ties_that_overflow_a_list(fa, dtype):
    """Borders that hundreds of tokens share, among others and alone."""
    g = gen(2)
    V = 20000
    x = torch.randn(6, V, generator=g) * 2
    x[0, ::10] = 3.0
    x[1, ::3] = 1.0
    x[2] = x[2].round()
    x[3] = 0.25
    x[4] = (x[4] * 4).round() / 4
    x[5, :600] = 9.0
    x = x.to(DT[dtype])
    u = us(6, g)
    check(fa, x, u, k=[900, 300, 150, 40, 384, 100])
    check(fa, x, u, p=[0.9, 0.6, 0.7, 0.31, 0.85, 0.43])
    check(fa, x, u, k=[5000, 7000, 9000, 19000, 12000, 590], p=[0.77, 0.9, 0.95, 0.4703, 0.6, 0.99])


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
def test_borders_near_zero(fa, dtype):
    """Logits of every magnitude on both sides of 0: the keys between them are billions."""
    g = gen(3)
    V = 30000
    x = torch.randn(8, V, generator=g) * torch.exp2(-torch.randint(0, 20, (8, V), generator=g).float())
    x[1] *= 2.0 ** -3
    x[2] *= 2.0 ** -8
    x[3, 0] = 8.0
    x[4, ::2] = 0.0
    x[5, 1::2] = -0.0
    x = x.to(DT[dtype])
    u = us(8, g)
    for p in (0.3, 0.5, 0.62, 0.9, 0.999):
        check(fa, x, u, p=[p] * 8)
    check(fa, x, u, k=[15000] * 8)
    check(fa, x, u, k=[100] * 8, p=[0.4] * 8)


def test_subnormal_logits(fa):
    """They are told apart and are not 0 (temperatures at which it shows)."""
    g = gen(4)
    for dtype, unit in (("fp32", 2.0 ** -149), ("bf16", 2.0 ** -133), ("fp16", 2.0 ** -24)):
        x = (torch.randint(-7, 8, (4, 500), generator=g).double() * unit).to(DT[dtype])
        assert (x != 0).any()
        u = us(4, g)
        check(fa, x, u, T=[0.0] * 4)
        check(fa, x, u, k=[50] * 4)
        if dtype == "fp16":
            check(fa, x, u, T=[2.0 ** -23] * 4, k=[50] * 4, p=[0.9] * 4)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_few_finite_logits(fa, dtype):
    """A grammar that allows few tokens: -infinity, or the type's lowest value, elsewhere."""
    g = gen(5)
    V = 40000
    x = torch.full((9, V), float("-inf"))
    for r, n in enumerate([1, 2, 30, 400, 600, 5000, 30, 400, 5000]):
        if r >= 6:
            x[r] = torch.finfo(DT[dtype]).min
        x[r, torch.randperm(V, generator=g)[:n]] = torch.randn(n, generator=g) * 2
    x = x.to(DT[dtype])
    u = us(9, g)
    for k in (None, [50] * 9, [500] * 9, [4000] * 9):
        for p in (None, [0.9] * 9):
            check(fa, x, u, k=k, p=p)
            check(fa, x, u, k=k, p=p, m=[0.05] * 9)


@pytest.mark.parametrize("shift", [-9000.0, -40.0, 700.0, 1e5])
def test_logits_far_from_zero(fa, shift):
    g = gen(6)
    x = torch.randn(6, 12345, generator=g) * 2 + shift
    u = us(6, g)
    T = [0.05, 0.4, 1.0, 3.0, 50.0, 1e4]
    check(fa, x, u, T=T)
    check(fa, x, u, T=T, p=[0.8] * 6)
    check(fa, x, u, T=T, k=[77] * 6, m=[0.02] * 6)


def test_min_p_beside_top_p(fa):
    """min_p's border far above, near and below top_p's."""
    g = gen(7)
    x = torch.randn(12, 50000, generator=g) * 2
    u = us(12, g)
    p = [0.2, 0.5, 0.8, 0.95] * 3
    m = [0.5] * 4 + [0.05] * 4 + [0.0001] * 4
    check(fa, x, u, p=p, m=m)
    check(fa, x.bfloat16(), u, T=[0.6] * 12, p=p, m=m)
    check(fa, x, u, m=[1.0, 0.999, 2.0, 1e-30, 1e-45, 0.9] * 2)


@pytest.mark.parametrize("p", [1e-6, 0.001, 0.9999, 0.99999])
def test_extreme_top_p(fa, p):
    g = gen(8)
    for sharp in (0.01, 1.0, 6.0):
        x = torch.randn(3, 33333, generator=g) * sharp
        check(fa, x, us(3, g), p=[p] * 3)


def test_more_rows_than_fit_at_once(fa):
    g = gen(9)
    R = 1300
    x = (torch.randn(R, 700, generator=g) * 2).half()
    k = torch.randint(0, 90, (R,), generator=g).tolist()
    p = (0.5 + 0.6 * torch.rand(R, generator=g)).tolist()
    check(fa, x, us(R, g), k=k, p=p)


@pytest.mark.parametrize("dtype,V", [("fp32", 360445), ("bf16", 720889), ("fp16", 600001)])
def test_largest_vocabularies(fa, dtype, V):
    g = gen(10)
    x = (torch.randn(2, V, generator=g) * 2).to(DT[dtype])
    u = us(2, g)
    check(fa, x, u, T=[0.8, 1.2], p=[0.9, 0.95])
    check(fa, x, u, k=[200, 5000], m=[0.001, 0.0])


def test_refuses_what_eight_sms_do_not_hold(fa):
    u = torch.zeros(1, device="cuda")
    for dtype, V in ((torch.float32, 360446), (torch.bfloat16, 720890)):
        with pytest.raises(fa.FAError) as e:
            fa.sample(torch.zeros(1, V, dtype=dtype, device="cuda"), u)
        assert e.value.status == fa.FA_ERR_UNSUPPORTED


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
def test_nan_and_zeros_of_both_signs(fa, dtype):
    """NaN of either sign counts as -infinity; -0 and 0 are equal, and go by index."""
    g = gen(11)
    V = 3000
    x = torch.randn(6, V, generator=g)
    x[0, ::3] = float("nan")
    x[1, 1::2] = -float("nan")
    x[2] = torch.where(torch.rand(V, generator=g) < 0.5, 0.0, -0.0)
    x[3] = torch.where(torch.rand(V, generator=g) < 0.5, 0.0, -0.0)
    x[3, ::7] = -1.0
    x[4, ::2] = float("inf")
    x[4, 1::4] = float("nan")
    x[5] = float("nan")
    x[5, 2222] = -3.0
    x = x.to(DT[dtype])
    assert torch.signbit(x[2]).any() and x.isnan().any()
    u = us(6, g)
    for k in (None, [100] * 6, [1401] * 6):
        for p in (None, [0.71313] * 6):
            check(fa, x, u, k=k, p=p)
            check(fa, x, u, T=[0.0] * 6, k=k, p=p)


def test_long_lists_again_and_again(fa):
    """Rows whose list overflows, so that the border comes from counts: many at once, many
    times, always the tokens that the order says."""
    g = gen(12)
    R, V, k = 600, 777, 166
    x = (torch.randn(R, V, generator=g) * 2).round() / 2
    x = x.half()
    u = torch.rand(R, generator=g).cuda()
    ks = torch.full((R,), k, dtype=torch.int32, device="cuda")
    order = torch.sort(x.float(), dim=-1, descending=True, stable=True).indices
    want = torch.zeros(R, V, dtype=torch.bool).scatter_(-1, order[:, :k], True).cuda()
    xd = x.cuda()
    first = None
    for _ in range(60):
        tok, probs = fa.sample(xd, u, top_k=ks, probs=True)
        assert torch.equal(probs > 0, want)
        first = tok if first is None else first
        assert torch.equal(tok, first)
