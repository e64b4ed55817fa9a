"""The draft-tree operators together, as a decoding step uses them: the drafted
tokens' keys and values normed, rotated and written to the cache pages, the
tree's attention, the verification and the compaction; eagerly, captured in a
graph and replayed, as two graphs at once, and with waits that run out."""
import random

import numpy as np
import pytest
import torch

from tests import tree_plain as tp

pytestmark = pytest.mark.gpu
EPS = 1e-5


class Step:
    """Device buffers of one decoding step of B sequences over two layers."""

    def __init__(self, B, N, Hq, Hkv, D, V, page, max_pages, seed, dtype=torch.bfloat16):
        g = torch.Generator().manual_seed(seed)
        self.B, self.N, self.Hq, self.Hkv, self.D, self.V, self.page = B, N, Hq, Hkv, D, V, page
        self.g, self.rng, self.dtype = g, random.Random(seed), dtype
        P = B * max_pages + 2
        self.kp = torch.full((2, P, page, Hkv, D), float("nan"), dtype=dtype, device="cuda")
        self.vp = self.kp.clone()
        self.table = torch.randperm(P, generator=g)[:B * max_pages].reshape(B, max_pages).int().cuda()
        self.lens = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.qw, self.kw = [(1 + 0.2 * torch.randn(D, generator=g)).to(dtype).cuda() for _ in range(2)]
        i = torch.arange(D // 2, dtype=torch.float64)
        self.freq = (10000.0 ** (-2 * i / D)).float().cuda()
        self.qkv = torch.zeros(2, B, N, Hq + 2 * Hkv, D, dtype=dtype, device="cuda")
        self.parents = torch.zeros(B, N, dtype=torch.int32, device="cuda")
        self.pos = torch.zeros(B, N, dtype=torch.int32, device="cuda")
        self.p = torch.zeros(B, N, V, device="cuda")
        self.q = torch.zeros(B, N, V, device="cuda")
        self.tokens = torch.zeros(B, N, dtype=torch.int32, device="cuda")
        self.u = torch.zeros(B, N, device="cuda")

    def draw(self, lens):
        """New inputs, in place.  lens: lengths with the tree's slots."""
        B, N, V, g = self.B, self.N, self.V, self.g
        par = tp.random_parents(B, N, self.rng)
        depth = [[0] * N for _ in range(B)]
        for b in range(B):
            for s in range(1, N):
                depth[b][s] = depth[b][par[b][s]] + 1
        self.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        self.parents.copy_(torch.tensor(par, dtype=torch.int32))
        self.pos.copy_(torch.tensor([[L - N + d for d in ds] for L, ds in zip(lens, depth)],
                                    dtype=torch.int32))
        self.qkv.copy_(torch.randn(self.qkv.shape, generator=g).to(self.dtype))
        lg = torch.randn(B, N, V, generator=g) * 1.5
        p = torch.softmax(lg, -1)
        q = torch.softmax(lg + 0.5 * torch.randn(B, N, V, generator=g), -1)
        tok = [[int(torch.multinomial(q[b, max(par[b][s], 0)], 1, generator=g)) for s in range(N)]
               for b in range(B)]
        self.p.copy_(p)
        self.q.copy_(q)
        self.tokens.copy_(torch.tensor(tok, dtype=torch.int32))
        self.u.copy_(torch.rand(B, N, generator=g))

    def run(self, fa, stream=None):
        Hq, Hkv = self.Hq, self.Hkv
        outs = []
        for layer in range(2):
            x = self.qkv[layer]
            q = fa.qk_norm_rope_append(x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:], self.qw,
                                       self.kw, self.freq, self.kp[layer], self.vp[layer], self.table,
                                       self.lens, EPS, positions=self.pos, stream=stream)
            outs.append((q,) + fa.decode_tree(q, self.kp[layer], self.vp[layer], self.table, self.lens,
                                              self.parents, self.D ** -0.5, lse=True, stream=stream))
        path, count, nxt = fa.verify_tree(self.p, self.q, self.tokens, self.parents, self.u,
                                          stream=stream)
        new = fa.compact_tree(self.kp, self.vp, self.table, self.lens, path, count, stream=stream)
        return outs, path, count, nxt, new


def check_step(st, before, out):
    """One step's outputs against the plain forms; ``before``: the pools as
    they were.  Returns the new lengths."""
    outs, path, count, nxt, new = out
    Hq, Hkv, N, page = st.Hq, st.Hkv, st.N, st.page
    lens, table = st.lens.tolist(), st.table.cpu().numpy()
    ang = tp.angles(st.pos.cpu().numpy(), st.freq)
    want_lens = None
    for layer in range(2):
        x = st.qkv[layer]
        q, o, lse = outs[layer]
        tp.check_rope(q, x[:, :, :Hq], st.qw, ang, EPS, False)
        # The tree's rows as the append left them: the compaction has moved some
        # of them, so they are written again, from the library's own outputs of
        # the rotation (checked above for q; k goes the same way).
        k, v = before[0][layer].clone(), before[1][layer].clone()
        ref, size = tp.norm_rope(x[:, :, Hq:Hq + Hkv], st.kw, ang, EPS, False)
        for b, L in enumerate(lens):
            for s in range(N):
                t = L - N + s
                k[table[b, t // page], t % page] = torch.from_numpy(ref[b, s]).to(k.dtype)
                v[table[b, t // page], t % page] = x[b, s, Hq + Hkv:].cpu()
        # (k here is the 64-bit key rounded once; the kernel's may differ by a
        # rounding, a relative 2^-7 of single elements, which check_tree's bound
        # on the scores takes in through a wider E.)
        O, ref_lse, A, E = tp.decode_tree(q, k, v, table, lens, st.parents.tolist(), st.D ** -0.5)
        err = np.abs(tp.f64(o) - O)
        assert np.isfinite(tp.f64(o)).all()
        assert np.all(err <= 2.0 ** -8 * 1.01 * (A + np.abs(O)) + 0.06 * A)
        pool_k, pool_v = k[None], v[None]
        for pool, dev in ((pool_k, st.kp), (pool_v, st.vp)):
            want_lens = tp.compact(pool, table, lens, path.tolist(), count.tolist(), N)
            got = dev[layer].cpu()
            for b, L in enumerate(want_lens):
                for t in range(L):
                    a, c = got[table[b, t // page], t % page], pool[0, table[b, t // page], t % page]
                    if dev is st.vp:
                        assert torch.equal(a, c)
                    else:
                        assert (a.float() - c.float()).abs().max() <= 2.0 ** -7 * c.float().abs().max()
    for b in range(st.B):
        way, tok = tp.verify(st.p[b].cpu().numpy(), st.q[b].cpu().numpy(), st.tokens[b].tolist(),
                             st.parents[b].tolist(), st.u[b].tolist())
        assert path[b].tolist() == way + [-1] * (N - len(way))
        assert int(count[b]) == len(way) and int(nxt[b]) == tok
    assert new.tolist() == want_lens
    return want_lens


def pools(st):
    return st.kp.cpu(), st.vp.cpu()


@pytest.mark.parametrize("stream", [False, True])
def test_three_steps(fa, stream):
    """Committed lengths grow by what was accepted; each step sees the rows that
    the last one kept.  (Every slot starts as NaN: a row that was never written
    would show.)"""
    st = Step(B=3, N=7, Hq=4, Hkv=2, D=64, V=24, page=32, max_pages=3, seed=1)
    side = torch.cuda.Stream() if stream else None
    lens = [0, 0, 0]
    for _ in range(3):
        st.draw([L + st.N for L in lens])
        before = pools(st)
        if side:
            side.wait_stream(torch.cuda.current_stream())
        out = st.run(fa, side)
        torch.cuda.synchronize()
        assert fa.fa_device_error()[0] == fa.FA_OK
        lens = check_step(st, before, out)
    assert min(lens) >= 3 and max(lens) > 3


def test_captured_and_replayed(fa):
    """One capture, replayed on new inputs and lengths."""
    st = Step(B=2, N=9, Hq=8, Hkv=2, D=128, V=40, page=64, max_pages=2, seed=2)
    st.draw([9, 9])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        st.run(fa)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = st.run(fa)
    lens = [0, 0]
    for _ in range(3):
        st.draw([L + st.N for L in lens])
        before = pools(st)
        graph.replay()
        torch.cuda.synchronize()
        assert fa.fa_device_error()[0] == fa.FA_OK
        lens = check_step(st, before, out)


def test_two_graphs_at_once(fa):
    """Two captured steps replayed side by side on two streams, many times: no
    scratch is shared between them, so each repeats its own bits."""
    steps, graphs, outs, refs = [], [], [], []
    for seed in (3, 4):
        st = Step(B=4, N=24, Hq=32, Hkv=2, D=128, V=5000, page=64, max_pages=8, seed=seed)
        st.kp.normal_()
        st.vp.normal_()
        st.draw([24 + 100 * (b + 1) for b in range(4)])
        keep = st.kp.clone(), st.vp.clone()
        refs.append(st.run(fa))
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=side):
            st.kp.copy_(keep[0])
            st.vp.copy_(keep[1])
            outs.append(st.run(fa))
        steps.append((st, side))
        graphs.append(gr)
    torch.cuda.synchronize()
    for _ in range(20):
        for gr, (_, side) in zip(graphs, steps):
            with torch.cuda.stream(side):
                gr.replay()
    torch.cuda.synchronize()
    assert fa.fa_device_error()[0] == fa.FA_OK
    for ref, out in zip(refs, outs):
        for a, b in zip(ref[0], out[0]):
            for x, y in zip(a, b):
                assert torch.equal(x, y)
        for x, y in zip(ref[1:], out[1:]):
            assert torch.equal(x, y)


def test_eager_streams_do_not_share_scratch(fa):
    """Tree decodes and gradients of the rotation in flight on several streams
    at once: each gives the bits it gives alone."""
    st = Step(B=2, N=16, Hq=16, Hkv=2, D=64, V=8, page=64, max_pages=30, seed=5)
    st.kp.normal_()
    st.vp.normal_()
    st.draw([1900, 1500])
    q = torch.randn(2, 16, 16, 64, device="cuda").to(st.dtype)
    x = torch.randn(3000, 20, 64, device="cuda").to(st.dtype)
    pos = torch.arange(3000, dtype=torch.int32, device="cuda")
    w = torch.ones(64, dtype=st.dtype, device="cuda")
    gq, gk = x[:, 2:18].contiguous(), x[:, :2].contiguous()

    def calls(s=None):
        a = fa.decode_tree(q, st.kp[0], st.vp[0], st.table, st.lens, st.parents, 0.1, lse=True, stream=s)
        b = fa.qk_norm_rope_backward(gq, gk, x[:, :16], x[:, 16:18], w, w, st.freq, pos, EPS, stream=s)
        return list(a) + list(b)

    ref = calls()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    got = []
    for _ in range(5):
        for s in streams:
            got.append(calls(s))
    torch.cuda.synchronize()
    for g in got:
        for a, b in zip(ref, g):
            assert torch.equal(a, b)


def test_threads_call_at_once(fa):
    """Four threads, a stream each, with calls of every operator in flight: each
    gives the bits it gives alone."""
    import threading
    steps, refs = [], []
    for seed in range(4):
        st = Step(B=2, N=12, Hq=16, Hkv=2, D=64, V=3000, page=64, max_pages=12, seed=20 + seed)
        st.kp.normal_()
        st.vp.normal_()
        st.draw([700 - 50 * seed, 300])
        st.keep = st.kp.clone(), st.vp.clone()
        refs.append(st.run(fa))
        steps.append(st)
    torch.cuda.synchronize()
    got = [None] * 4

    def work(i):
        st, mine = steps[i], []
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(10):
                st.kp.copy_(st.keep[0])
                st.vp.copy_(st.keep[1])
                mine.append(st.run(fa))
        got[i] = mine

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert fa.fa_device_error()[0] == fa.FA_OK
    for ref, mine in zip(refs, got):
        for out in mine:
            for a, b in zip(ref[0], out[0]):
                for x, y in zip(a, b):
                    assert torch.equal(x, y)
            for x, y in zip(ref[1:], out[1:]):
                assert torch.equal(x, y)


def test_streams_given_as_handles(fa):
    """A stream as torch's object, as its handle, and as the handles of the null
    and the legacy stream."""
    st = Step(B=1, N=5, Hq=4, Hkv=2, D=64, V=50, page=32, max_pages=2, seed=30)
    st.kp.normal_()
    st.vp.normal_()
    st.draw([40])
    q = torch.randn(1, 5, 4, 64, device="cuda").to(st.dtype)
    args = (q, st.kp[0], st.vp[0], st.table, st.lens, st.parents, 0.125)
    ref = fa.decode_tree(*args)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for s in (side, side.cuda_stream, 0, 1, 2):  # (1: the legacy stream, 2: the thread's own)
        out = fa.decode_tree(*args, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(out, ref), s


def test_call_from_a_new_thread(fa):
    """A thread that has made no CUDA call yet, with outputs that are there."""
    import threading
    st = Step(B=1, N=5, Hq=4, Hkv=2, D=64, V=50, page=32, max_pages=2, seed=31)
    st.kp.normal_()
    st.vp.normal_()
    st.draw([40])
    q = torch.randn(1, 5, 4, 64, device="cuda").to(st.dtype)
    args = (q, st.kp[0], st.vp[0], st.table, st.lens, st.parents, 0.125)
    ref, out, side, errors = fa.decode_tree(*args), torch.empty_like(q), torch.cuda.Stream(), []
    torch.cuda.synchronize()

    def call():
        try:
            fa.decode_tree(*args, out=out, stream=side)
        except Exception as e:
            errors.append(e)

    t = threading.Thread(target=call)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    assert torch.equal(out, ref)


def test_first_call_while_another_thread_captures():
    """What the first call sets up (the kernels' module and attributes, the
    scratch pool), here while a capture that forbids such calls on every thread
    is under way: the capture goes on, and both results are right.  (A process
    of its own: it is set up once.)"""
    import subprocess
    import sys
    code = """
import threading, torch
import attention_fa_fwd_04_gb300 as fa
bf, i32 = torch.bfloat16, torch.int32
g = torch.Generator().manual_seed(1)
q = torch.randn(1, 4, 4, 64, generator=g).to(bf).cuda()
kp, vp = (torch.randn(9, 32, 2, 64, generator=g).to(bf).cuda() for _ in range(2))
table = torch.arange(9, dtype=i32, device="cuda")[None]
lens = torch.tensor([280], dtype=i32, device="cuda")
parents = torch.tensor([[-1, 0, 0, 2]], dtype=i32, device="cuda")
out, x = torch.empty_like(q), torch.ones(8, device="cuda")
side, errors = torch.cuda.Stream(), []
torch.cuda.synchronize()
def other():
    try:
        fa.decode_tree(q, kp, vp, table, lens, parents, 0.125, out=out, stream=side)
    except Exception as e:
        errors.append(e)
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph, capture_error_mode="global"):
    x.mul_(2)
    t = threading.Thread(target=other)
    t.start()
    t.join()
    x.add_(1)
graph.replay()
torch.cuda.synchronize()
assert not errors, errors
assert x.tolist() == [3.0] * 8
assert torch.equal(out, fa.decode_tree(q, kp, vp, table, lens, parents, 0.125))
assert fa.fa_device_error()[0] == fa.FA_OK
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_waits_that_run_out_report_and_the_next_calls_are_correct(fa):
    """A limit of 1 ns: the norm and rotation and the tree decode (its loader
    polls for ring slots) give up, report FA_ERR_TIMEOUT and return; at the
    default limit the next step is right.
    (The rotation's gradient has the forward's waits, but more arithmetic than
    its loads take: they need not run out, so either answer will do.)"""
    st = Step(B=2, N=8, Hq=8, Hkv=2, D=128, V=4000, page=64, max_pages=2, seed=6)
    st.draw([120, 90])
    # 336 MB, past the 129 MB of L2: the rotation's loads are slower than its
    # arithmetic, so its rings run dry.  (42 MB that were just written do not.)
    big = torch.empty(32768, 40, 128, dtype=st.dtype, device="cuda").normal_()
    pos = torch.arange(32768, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    assert fa.fa_device_error()[0] == fa.FA_OK
    calls = [
        lambda: fa.qk_norm_rope(big[:, :32], big[:, 32:], st.qw, st.kw, st.freq, pos, EPS),
    ]
    # 78000 keys of 2 kv heads are 1220 tiles, eight or nine for each of 152
    # CTAs, whose rings hold three: the loader waits.
    tq = big[:16, :8].reshape(2, 8, 8, 128).contiguous()
    long = Step(B=2, N=8, Hq=8, Hkv=2, D=128, V=8, page=64, max_pages=630, seed=9)
    long.kp.normal_()
    long.vp.normal_()
    long.draw([40000, 38000])
    calls.append(lambda: fa.decode_tree(tq, long.kp[0], long.vp[0], long.table, long.lens, long.parents,
                                        0.1))
    try:
        assert fa.fa_set_wait_limit_ns(1) == fa.FA_OK
        for call in calls:
            call()
            st_, detail = fa.fa_device_error()
            assert st_ == fa.FA_ERR_TIMEOUT, (calls.index(call), hex(detail))
            assert (detail >> 16) & 1 and (detail >> 24) & 0xFF, hex(detail)
        fa.qk_norm_rope_backward(big[:, :32].contiguous(), big[:, 32:].contiguous(), big[:, :32],
                                 big[:, 32:], st.qw, st.kw, st.freq, pos, EPS)
        assert fa.fa_device_error()[0] in (fa.FA_OK, fa.FA_ERR_TIMEOUT)
    finally:
        assert fa.fa_set_wait_limit_ns(0) == fa.FA_OK
    small = Step(B=2, N=5, Hq=4, Hkv=2, D=64, V=24, page=32, max_pages=2, seed=7)
    small.draw([5, 5])
    before = pools(small)
    out = small.run(fa)
    torch.cuda.synchronize()
    assert fa.fa_device_error()[0] == fa.FA_OK
    check_step(small, before, out)


def test_prefill_of_normed_heads(fa):
    """The rotation's outputs feed the prefill, and the gradients chain back:
    prefill(qk_norm_rope(q, k)) and its backward against the 64-bit oracle of
    the attention on the library's own rotated heads."""
    import oracle
    from tests.parity import compare
    B, S, Hq, Hkv, D = 1, 300, 4, 2, 64
    g = torch.Generator().manual_seed(8)
    qkv = torch.randn(B, S, Hq + 2 * Hkv, D, generator=g).bfloat16().cuda()
    w = (1 + 0.1 * torch.randn(D, generator=g)).bfloat16().cuda()
    f = (10000.0 ** (-torch.arange(32, dtype=torch.float64) / 32)).float().cuda()
    pos = torch.arange(S, dtype=torch.int32, device="cuda")[None]
    q, k = fa.qk_norm_rope(qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], w, w, f, pos, EPS)
    v = qkv[:, :, Hq + Hkv:].contiguous()
    o, lse = fa.prefill(q, k, v, 0.125, True, lse=True)
    do = torch.randn(o.shape, generator=g).bfloat16().cuda()
    dq, dk, dv = fa.backward(q, k, v, o, do, lse, 0.125, True)
    gq, gk, gqw, gkw = fa.qk_norm_rope_backward(dq, dk, qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], w, w, f,
                                                pos, EPS)
    torch.cuda.synchronize()
    assert fa.fa_device_error()[0] == fa.FA_OK
    compare(o.float().cpu().numpy(), oracle.attention(q.cpu(), k.cpu(), v.cpu(), 0.125, True))
    ang = tp.angles(pos.cpu().numpy(), f)
    for x, gr, dx in ((qkv[:, :, :Hq], dq, gq), (qkv[:, :, Hq:Hq + Hkv], dk, gk)):
        ref, _, size, _ = tp.norm_rope_grad(x, w, gr, ang, EPS, False)
        assert np.all(np.abs(tp.f64(dx) - ref) <= 2.0 ** -8 * np.abs(ref) + 97 * tp.U32 * size)


def run_keeping(st, fa):
    """A step, and the pools as its attention read them: behind the appends and
    before the compaction."""
    append, compact, kept = fa.qk_norm_rope_append, fa.compact_tree, []

    class Calls:
        qk_norm_rope_append = staticmethod(append)
        decode_tree = staticmethod(fa.decode_tree)
        verify_tree = staticmethod(fa.verify_tree)

        @staticmethod
        def compact_tree(*a, **kw):
            kept.extend((st.kp.clone(), st.vp.clone()))
            return compact(*a, **kw)

    return st.run(Calls), kept


def check_attention(st, out, kept):
    """O and log-sum-exp on the library's own keys, to check_tree's bounds, and the
    keys themselves to the rotation's."""
    Hq, Hkv, N, page = st.Hq, st.Hkv, st.N, st.page
    lens, table = st.lens.tolist(), st.table.cpu().numpy()
    ang = tp.angles(st.pos.cpu().numpy(), st.freq)
    for layer in range(2):
        q, o, lse = out[0][layer]
        k, v, x = kept[0][layer].cpu(), kept[1][layer].cpu(), st.qkv[layer].cpu()
        tp.check_tree(o, lse, q, k, v, table, lens, st.parents.tolist(), st.D ** -0.5)
        for b, L in enumerate(lens):
            t = np.arange(L - N, L)
            rows = table[b, t // page], t % page
            tp.check_rope(k[rows], x[b, :, Hq:Hq + Hkv], st.kw, ang[b], EPS, False)
            assert torch.equal(v[rows], x[b, :, Hq + Hkv:])


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("B,N,Hq,Hkv,D,page,max_pages,dtype", [
    (3, 7, 4, 2, 64, 32, 6, torch.bfloat16),
    (2, 9, 8, 2, 128, 64, 5, torch.float16),
    (2, 40, 16, 2, 64, 96, 4, torch.bfloat16),   # 320 rows: three row tiles
    (1, 64, 8, 2, 128, 64, 6, torch.bfloat16),   # 256 rows: two
])
def test_attention_of_steps_to_its_own_bounds(fa, B, N, Hq, Hkv, D, page, max_pages, dtype, captured):
    """Steps over changing lengths, in which a wrong mask, length or row shows in
    the log-sum-exp (test_tree_check.py plants some)."""
    st = Step(B, N, Hq, Hkv, D, 24, page, max_pages, seed=B + N + D, dtype=dtype)
    st.draw([N] * B)
    run_keeping(st, fa)  # (set-up)
    torch.cuda.synchronize()
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out, kept = run_keeping(st, fa)
    # A prompt of other lengths in each sequence.
    st.kp.fill_(float("nan"))
    st.vp.fill_(float("nan"))
    lens = [(37 * b + 51) % (max_pages * page - 4 * N) for b in range(B)]
    for b, L in enumerate(lens):
        t = np.arange(L)
        rows = torch.from_numpy(st.table.cpu().numpy()[b, t // page]).long().cuda(), torch.from_numpy(t % page).cuda()
        for pool in (st.kp, st.vp):
            for layer in range(2):
                pool[layer][rows] = torch.randn(L, Hkv, D, generator=st.g).to(dtype).cuda()
    for _ in range(3):
        st.draw([L + N for L in lens])
        if captured:
            graph.replay()
        else:
            out, kept = run_keeping(st, fa)
        torch.cuda.synchronize()
        assert fa.fa_device_error()[0] == fa.FA_OK
        check_attention(st, out, kept)
        lens = out[4].tolist()


def test_kept_scratch_is_given_back(fa):
    """fa_release_scratch: what a call freed goes back to the driver; calls before
    and behind it are as ever, one in flight among them."""
    st = Step(B=4, N=64, Hq=128, Hkv=8, D=128, V=8, page=64, max_pages=32, seed=40)
    st.kp.normal_()
    st.vp.normal_()
    st.draw([2000, 1900, 1500, 700])
    q = torch.randn(4, 64, 128, 128, device="cuda").to(st.dtype)
    args = (q, st.kp[0], st.vp[0], st.table, st.lens, st.parents, 0.088)
    ref = fa.decode_tree(*args)
    torch.cuda.synchronize()
    held = torch.cuda.mem_get_info()[0]
    assert fa.fa_release_scratch() == fa.FA_OK
    freed = torch.cuda.mem_get_info()[0] - held
    assert freed >= 2 ** 24  # (the partials: 152 CTAs x 2 x 256 rows x 130 floats = 40 MB)
    outs = []
    for _ in range(3):
        outs.append(fa.decode_tree(*args))
        assert fa.fa_release_scratch() == fa.FA_OK
    torch.cuda.synchronize()
    assert all(torch.equal(o, ref) for o in outs)
    assert fa.fa_device_error()[0] == fa.FA_OK
