"""The serving-step operators together, as a decoding step uses them: the page bookkeeping,
the new tokens' rows written to their slots, attention over the pages with a shared prefix,
the next tokens; eagerly, captured and replayed, as two graphs at once, from several
threads and streams, and with waits that run out."""
import random
import threading

import pytest
import torch

from tests import serving_plain as sp

pytestmark = pytest.mark.gpu


class Serving:
    """Device buffers of B sequences; the first `members` share `prefix` whole pages."""

    def __init__(self, B, Hq, Hkv, D, V, page, width, prefix, members, seed, spare=4, dtype=torch.bfloat16):
        g = torch.Generator().manual_seed(seed)
        self.g, self.rng = g, random.Random(seed)
        self.B, self.Hq, self.Hkv, self.D, self.V, self.page, self.width = B, Hq, Hkv, D, V, page, width
        self.members, self.max_new, self.dtype = members, 2 * page + B, dtype
        P = prefix + B * width // 2 + spare
        self.pages = P
        ids = torch.randperm(P, generator=g).tolist()
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        # (NaN where nothing has been written: a row read before its write would show.)
        self.kp = torch.full((P, page, Hkv, D), float("nan"), dtype=dtype, device="cuda")
        self.vp = self.kp.clone()
        for pid in ids[:prefix]:
            for pool in (self.kp, self.vp):
                pool[pid] = torch.randn(page, Hkv, D, generator=g).to(dtype)
        rows = [[ids[j] if b < members and j < prefix else 0 for j in range(width)] for b in range(B)]
        self.table = i32(rows)
        self.lens = i32([prefix * page if b < members else 0 for b in range(B)])
        self.shared = i32([prefix if b < members else 0 for b in range(B)])
        self.free = i32(ids[prefix:] + [0] * prefix)
        self.count = i32([P - prefix])
        self.starts, self.prefix = i32([0, members]), i32([prefix * page])
        self.new = torch.zeros_like(self.lens)
        self.kv = torch.zeros(self.max_new, 2 * Hkv, D, dtype=dtype, device="cuda")
        self.q = torch.zeros(B, 1, Hq, D, dtype=dtype, device="cuda")
        self.logits = torch.zeros(B, V, dtype=dtype, device="cuda")
        self.u, self.T, self.tp = (torch.zeros(B, device="cuda") for _ in range(3))
        self.k = torch.zeros(B, dtype=torch.int32, device="cuda")

    def draw(self):
        """The next step's inputs, in place: every sequence one token more, some prompts
        enter, some sequences leave (members back to the prefix)."""
        g, new = self.g, []
        for b, L in enumerate(self.lens.tolist()):
            base = int(self.prefix) if b < self.members else 0
            if L == base:
                L += self.rng.choice([0, 1, self.page // 2 + 1])
            elif self.rng.random() < 0.2 or L >= self.width * self.page:
                L = base
            else:
                L += 1
            new.append(L)
        self.new.copy_(torch.tensor(new, dtype=torch.int32))
        self.kv.copy_(torch.randn(self.kv.shape, generator=g).to(self.dtype))
        self.q.copy_(torch.randn(self.q.shape, generator=g).to(self.dtype))
        self.logits.copy_((torch.randn(self.logits.shape, generator=g) * 3).to(self.dtype))
        self.u.copy_(torch.rand(self.B, generator=g))
        self.T.copy_(0.5 + torch.rand(self.B, generator=g))
        self.tp.copy_(0.6 + 0.4 * torch.rand(self.B, generator=g))
        self.k.copy_(torch.randint(0, 30, (self.B,), generator=g, dtype=torch.int32))

    def run(self, fa, stream=None, in_place=True):
        lens, count, cu, slots, pos = fa.update_pages(
            self.table, self.lens, self.new, self.free, self.count, self.page, self.max_new,
            shared_pages=self.shared, lens_out=self.lens if in_place else None,
            free_count_out=self.count if in_place else None, stream=stream)
        fa.write_pages(self.kv[:, :self.Hkv], self.kv[:, self.Hkv:], self.kp, self.vp, slots, stream=stream)
        o, lse = fa.decode_shared(self.q, self.kp, self.vp, self.table, lens, self.starts, self.prefix,
                                  self.D ** -0.5, lse=True, stream=stream)
        tok, probs = fa.sample(self.logits, self.u, temperature=self.T, top_k=self.k, top_p=self.tp,
                               probs=True, stream=stream)
        return lens, count, cu, slots, pos, o, lse, tok, probs

    def state(self):
        return (self.table.tolist(), self.lens.tolist(), self.free.tolist(), int(self.count), self.kp.cpu(),
                self.vp.cpu())


def check(st, before, out):
    table, old, free, count, kp, vp = before
    lens, left, cu, slots, pos, o, lse, tok, probs = out
    want = sp.update_pages(table, old, st.new.tolist(), free, count, st.page, st.max_new, st.shared.tolist())
    assert not want[7]
    assert st.table.tolist() == want[0] and st.free.tolist() == want[1]
    assert lens.tolist() == want[2] and left.tolist() == [want[3]] and cu.tolist() == want[4]
    assert slots.tolist() == want[5] and pos.tolist() == want[6]
    kv = st.kv.cpu()
    for t, s in enumerate(want[5]):
        if s >= 0:
            kp[s // st.page, s % st.page] = kv[t, :st.Hkv]
            vp[s // st.page, s % st.page] = kv[t, st.Hkv:]
    for pool, dev in ((kp, st.kp), (vp, st.vp)):
        assert torch.equal(pool.view(torch.int16), dev.cpu().view(torch.int16))
    sp.check_decode(o, lse, st.q, kp, vp, torch.tensor(want[0]), want[2], st.D ** -0.5)
    rows = st.logits.float().cpu().double().numpy()
    for b in range(st.B):
        t, dist, margin = sp.sample(rows[b], float(st.u[b]), float(st.T[b]), int(st.k[b]), float(st.tp[b]))
        assert margin > 1e-9
        assert int(tok[b]) == t
        assert abs(probs[b].double().cpu().numpy() - dist).max() <= 2.0 ** -24 * 1.01


@pytest.mark.parametrize("stream", [False, True])
def test_steps(fa, stream):
    st = Serving(B=5, Hq=4, Hkv=2, D=64, V=300, page=32, width=5, prefix=2, members=3, seed=1)
    side = torch.cuda.Stream() if stream else None
    grown = 0
    for _ in range(6):
        st.draw()
        before = st.state()
        if side:
            side.wait_stream(torch.cuda.current_stream())
        out = st.run(fa, side)
        torch.cuda.synchronize()
        assert fa.fa_device_error()[0] == fa.FA_OK
        check(st, before, out)
        grown += int(out[2][-1])
    assert grown > 20


def test_captured_and_replayed(fa):
    """One capture; every replay takes the state that the last one left."""
    st = Serving(B=6, Hq=16, Hkv=2, D=128, V=1000, page=64, width=4, prefix=2, members=4, seed=2)
    st.draw()
    keep = [t.clone() for t in (st.table, st.lens, st.free, st.count, st.kp, st.vp)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = st.run(fa)
    for t, k in zip((st.table, st.lens, st.free, st.count, st.kp, st.vp), keep):
        assert torch.equal(t.nan_to_num() if t.is_floating_point() else t,
                           k.nan_to_num() if k.is_floating_point() else k)  # (nothing ran)
    for _ in range(5):
        st.draw()
        before = st.state()
        graph.replay()
        torch.cuda.synchronize()
        assert fa.fa_device_error()[0] == fa.FA_OK
        check(st, before, out)


def big(seed, fa=None):
    st = Serving(B=40, Hq=32, Hkv=4, D=128, V=20000, page=64, width=48, prefix=40, members=30, seed=seed)
    st.kp.normal_()
    st.vp.normal_()
    st.draw()
    return st


def test_two_graphs_at_once(fa):
    """Replayed side by side on two streams, many times: no scratch is shared between
    them, so each repeats its own bits."""
    steps, refs, outs = [], [], []
    for seed in (3, 4):
        st = big(seed)
        state = (st.table, st.free, st.kp, st.vp)
        keep = [t.clone() for t in state]
        refs.append([t.clone() for t in st.run(fa, in_place=False)])
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            for t, k in zip(state, keep):
                t.copy_(k)
            outs.append(st.run(fa, in_place=False))
        steps.append((st, side, graph, keep))
    torch.cuda.synchronize()
    for _ in range(20):
        for _, side, graph, _ in steps:
            with torch.cuda.stream(side):
                graph.replay()
    torch.cuda.synchronize()
    assert fa.fa_device_error()[0] == fa.FA_OK
    for ref, out in zip(refs, outs):
        for a, b in zip(ref, out):
            assert torch.equal(a, b)


def test_threads_with_streams_of_their_own(fa):
    """Calls of several threads in flight at once give the bits they give alone."""
    st = big(5)
    lens = torch.full((40,), 40 * 64, dtype=torch.int32, device="cuda") + torch.arange(
        40, dtype=torch.int32, device="cuda")
    lens[30:] = 777
    st.table.copy_(torch.randint(0, st.pages, st.table.shape, generator=st.g, dtype=torch.int32))
    st.table[1:30, :40] = st.table[0, :40]

    def calls():
        o = fa.decode_shared(st.q, st.kp, st.vp, st.table, lens, st.starts, st.prefix, 0.1, lse=True)
        return list(o) + list(fa.sample(st.logits, st.u, temperature=st.T, top_p=st.tp, probs=True))

    ref = [t.clone() for t in calls()]
    torch.cuda.synchronize()
    got, failed = [None] * 4, []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(10):
                    got[i] = calls()
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed
    assert fa.fa_device_error()[0] == fa.FA_OK
    for out in got:
        for a, b in zip(ref, out):
            assert torch.equal(a, b)


def test_outputs_given_and_scratch_released(fa):
    st = big(6)
    lens = torch.full((40,), 2000, dtype=torch.int32, device="cuda")
    st.table.copy_(torch.randint(0, st.pages, st.table.shape, generator=st.g, dtype=torch.int32))
    st.table[1:30, :40] = st.table[0, :40]
    lens[:30] += 1000
    ref = fa.decode_shared(st.q, st.kp, st.vp, st.table, lens, st.starts, st.prefix, 0.1, lse=True)
    out, lse = torch.empty_like(ref[0]), torch.empty_like(ref[1])
    torch.cuda.synchronize()
    assert fa.fa_release_scratch() == fa.FA_OK
    got = fa.decode_shared(st.q, st.kp, st.vp, st.table, lens, st.starts, st.prefix, 0.1, out=out, lse=lse)
    assert got[0].data_ptr() == out.data_ptr() and got[1].data_ptr() == lse.data_ptr()
    assert torch.equal(ref[0], out) and torch.equal(ref[1], lse)
    ref = fa.sample(st.logits, st.u, top_p=st.tp, probs=True)
    probs = torch.full_like(ref[1], -1.0)
    got = fa.sample(st.logits, st.u, top_p=st.tp, probs=probs)
    assert got[1].data_ptr() == probs.data_ptr()
    assert torch.equal(ref[0], got[0]) and torch.equal(ref[1], probs)


@pytest.mark.parametrize("Sq", [1, 4])
def test_waits_that_run_out(fa, Sq):
    """Under a limit of 1 ns the call ends and says so (rows streamed by warps beside the
    prefix's tiles, and all of them in tiles); the next call is right."""
    g = torch.Generator(device="cuda").manual_seed(8)
    B, Hq, Hkv, D, page, width = 12, 16, 2, 128, 64, 80
    kp = torch.randn(B * width, page, Hkv, D, device="cuda", generator=g).bfloat16()
    vp = torch.randn(B * width, page, Hkv, D, device="cuda", generator=g).bfloat16()
    q = torch.randn(B, Sq, Hq, D, device="cuda", generator=g).bfloat16()
    table = torch.arange(B * width, dtype=torch.int32, device="cuda").reshape(B, width)
    table[1:, :60] = table[0, :60]
    lens = torch.full((B,), width * page - 7, dtype=torch.int32, device="cuda")
    starts = torch.tensor([0, B], dtype=torch.int32, device="cuda")
    prefix = torch.tensor([60 * page], dtype=torch.int32, device="cuda")
    call = lambda: fa.decode_shared(q, kp, vp, table, lens, starts, prefix, D ** -0.5, lse=True)  # noqa: E731
    ref = call()
    torch.cuda.synchronize()
    assert fa.fa_device_error(reset=1)[0] == fa.FA_OK
    try:
        assert fa.fa_set_wait_limit_ns(1) == fa.FA_OK
        call()
        st, detail = fa.fa_device_error(reset=1)
    finally:
        assert fa.fa_set_wait_limit_ns(0) == fa.FA_OK
    assert st == fa.FA_ERR_TIMEOUT, (st, hex(detail))
    got = call()
    torch.cuda.synchronize()
    assert fa.fa_device_error(reset=1)[0] == fa.FA_OK
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
