"""Cases of the serving-step operators: a paged cache's bookkeeping, its rows, shared prefixes, sampling.

Four entry points of the binding are covered:

    decode_shared   attention of new tokens over a paged cache whose sequences share long prefixes
    sample          the next token from logits: temperature, top-k, top-p, min-p, a given uniform number
    update_pages    page table, free pages, slot map and positions from the sequences' old and new lengths
    write_pages     K and V rows of packed tokens into the cache's pages

``run`` computes them with elementary torch operations, or, where ``own`` is
true, through the binding.
"""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # A few users behind one system prompt, the single-token decode's heads: latency.
        dict(name="shared_small", op="shared", B=8, Sq=1, Hq=8, Hkv=2, D=128, dtype="bf16", groups=1,
             prefix=1500, own=200, page=64),
        # 64 chats behind one long system prompt.
        dict(name="shared_chat", op="shared", B=64, Sq=1, Hq=64, Hkv=8, D=128, dtype="bf16", groups=1,
             prefix=8192, own=1024, page=64),
        # 32 questions about one long document, the headline prefill's heads.
        dict(name="shared_document", op="shared", B=32, Sq=1, Hq=128, Hkv=8, D=128, dtype="bf16",
             groups=1, prefix=65536, own=2048, page=128),
        # Several prompts of odd lengths, four new tokens each, small fp16 heads, small pages.
        dict(name="shared_groups", op="shared", B=48, Sq=4, Hq=16, Hkv=4, D=64, dtype="fp16", groups=5,
             prefix=5001, own=333, page=32),
        # One user's token: latency.
        dict(name="sample_one", op="sample", B=1, V=32000, dtype="fp32", top_k=True, top_p=True,
             min_p=False, probs=False),
        # 64 users, each with settings of their own, a large vocabulary.
        dict(name="sample_batch", op="sample", B=64, V=128000, dtype="bf16", top_k=False, top_p=True,
             min_p=True, probs=False),
        # Temperature alone, odd vocabulary.
        dict(name="sample_plain", op="sample", B=200, V=50257, dtype="fp16", top_k=False, top_p=False,
             min_p=False, probs=False),
        # Distributions after 32 drafted nodes of 16 users, for their verification.
        dict(name="sample_probs", op="sample", B=512, V=32000, dtype="fp32", top_k=True, top_p=True,
             min_p=False, probs=True),
        # One more token for each of 64 sequences: latency.
        dict(name="pages_step", op="pages", B=64, page=64, max_pages=128, prompt=0, finish=0.0),
        # New prompts enter while other sequences leave.
        dict(name="pages_prompts", op="pages", B=256, page=64, max_pages=1024, prompt=1024, finish=0.2),
        # The K/V rows of one token per user: latency.
        dict(name="write_token", op="write", T=64, Hkv=2, D=128, dtype="bf16", page=64, packed=True),
        # The rows of a step's prompts.
        dict(name="write_prompt", op="write", T=65536, Hkv=8, D=128, dtype="bf16", page=64, packed=True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["shared", "shared", "shared", "sample", "sample", "pages", "write"])
    D, page = rng.choice([64, 128]), rng.choice([32, 64, 96, 128, 256])
    dtype = rng.choice(["bf16", "fp16"])
    Hkv = rng.choice([1, 2, 4, 5, 8, 16])
    G = rng.choice([1, 2, 3, 4, 7, 8, 16])
    while Hkv * G > 128:
        G = rng.choice([1, 2, 3, 4, 7, 8])
    if op == "shared":
        B = _log(rng, 2, 128)
        Sq = rng.choice([1, 1, 1, 2, 3, 4, 8])
        groups = _log(rng, 1, max(1, B // 2))
        rows, cache = 65536 * 32 * 128 // max(B * Sq * Hkv * G, 1024), 65536 * 8 * 128 // (Hkv * D)
        return dict(op=op, B=B, Sq=Sq, Hq=Hkv * G, Hkv=Hkv, D=D, dtype=dtype, groups=groups,
                    prefix=_log(rng, 16, min(65536, rows, cache // groups)),
                    own=_log(rng, Sq, max(Sq, min(4096, rows // 2, cache // B))), page=page)
    if op == "sample":
        V = _log(rng, 1000, 160000)
        return dict(op=op, B=_log(rng, 1, max(1, min(512, 512 * 32000 // V))), V=V,
                    dtype=rng.choice(["bf16", "fp16", "fp32"]), top_k=rng.random() < 0.5,
                    top_p=rng.random() < 0.6, min_p=rng.random() < 0.4, probs=rng.random() < 0.4)
    if op == "pages":
        max_pages = _log(rng, 8, 1024)
        most = max_pages * page // 2
        return dict(op=op, B=_log(rng, 1, 256), page=page, max_pages=max_pages,
                    prompt=rng.choice([0, _log(rng, 8, min(1024, most))]),
                    finish=rng.choice([0.0, 0.1, 0.3]))
    return dict(op=op, T=_log(rng, 1, min(65536, 65536 * 8 * 128 // (Hkv * D))), Hkv=Hkv, D=D, dtype=dtype,
                page=page, packed=rng.random() < 0.5)


# ----------------------------------------------------------------------------
# Sizes that a case's data lead to
# ----------------------------------------------------------------------------
def _shared_lengths(case):
    """Group starts, prefix lengths (the first the longest, the rest down to a quarter), own lengths."""
    B, n, P, own_most, Sq = case["B"], case["groups"], case["prefix"], case["own"], case["Sq"]
    rng = random.Random("%d %d %d" % (B, n, P))
    starts = [0] + sorted(rng.sample(range(1, B), n - 1)) + [B]
    prefix = [P if g == 0 else rng.randint(max(1, P // 4), P) for g in range(n)]
    tails = [own_most if b == 0 else rng.randint(max(Sq, own_most // 4), own_most) for b in range(B)]
    return starts, prefix, tails


def _page_lengths(case):
    """Old and new lengths: sequences that finish, that start with a prompt, that go on by a token."""
    B, cap = case["B"], case["max_pages"] * case["page"]
    rng = random.Random("%d %d %d" % (B, cap, case["prompt"]))
    old, new = [], []
    for _ in range(B):
        at = rng.randint(1, cap // 2)
        kind = rng.random()
        if kind < case["finish"]:
            old.append(at)
            new.append(0)
        elif case["prompt"] and kind < case["finish"] + 0.25:
            old.append(0)
            new.append(rng.randint(max(1, case["prompt"] // 4), case["prompt"]))
        else:
            old.append(at)
            new.append(at + 1)
    return old, new


def work(case):
    op = case["op"]
    if op == "shared":
        starts, prefix, tails = _shared_lengths(case)
        Sq, Hq, Hkv, D = case["Sq"], case["Hq"], case["Hkv"], case["D"]
        rows = case["B"] * Sq * Hq
        seen = sum(P * (starts[g + 1] - starts[g]) for g, P in enumerate(prefix)) + sum(tails)
        return {"bytes": (sum(prefix) + sum(tails)) * Hkv * D * 4 + rows * (D * 4 + 4),
                "flops": 4.0 * seen * Sq * Hq * D}
    if op == "sample":
        n = case["B"] * case["V"]
        return {"bytes": n * (4 if case["dtype"] == "fp32" else 2) + (n * 4 if case["probs"] else 0),
                "flops": n * 4}
    if op == "pages":
        old, new = _page_lengths(case)
        page = case["page"]
        tokens = sum(max(0, n - o) for o, n in zip(old, new))
        moved = sum(abs(-(-n // page) - -(-o // page)) for o, n in zip(old, new))
        return {"bytes": case["B"] * 16 + tokens * 8 + moved * 8, "flops": tokens * 2}
    return {"bytes": case["T"] * (case["Hkv"] * case["D"] * 8 + 4), "flops": 0}


# ----------------------------------------------------------------------------
# Inputs
# ----------------------------------------------------------------------------
def prepare(case, seed):
    rng = random.Random(seed)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, st = case["op"], {"case": case}

    def randn(*shape, dtype=None):
        return torch.empty(shape, dtype=dtype or DTYPES[case["dtype"]], device="cuda").normal_(generator=g)

    def rand(*shape):
        return torch.rand(*shape, device="cuda", generator=g)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    if op == "sample":
        B, V = case["B"], case["V"]
        st["logits"] = randn(B, V).mul_(2.5)
        st["u"] = rand(B)
        st["temperature"] = torch.where(rand(B) < 0.1, torch.zeros(B, device="cuda"), 0.5 + rand(B))
        k = torch.randint(1, 200, (B,), device="cuda", generator=g, dtype=torch.int32)
        st["top_k"] = torch.where(rand(B) < 0.2, torch.zeros_like(k), k) if case["top_k"] else None
        st["top_p"] = (0.7 + 0.4 * rand(B)).clamp(max=1.0) if case["top_p"] else None
        st["min_p"] = (0.15 * rand(B) - 0.03).clamp(min=0.0) if case["min_p"] else None
        return st
    page = case["page"]
    if op == "pages":
        old, new = _page_lengths(case)
        B, max_pages = case["B"], case["max_pages"]
        need = [-(-x // page) for x in old]
        total = sum(need) + sum(max(0, -(-n // page) - m) for n, m in zip(new, need)) + 64
        ids = list(range(total))
        rng.shuffle(ids)
        table = np.zeros((B, max_pages), np.int32)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = ids[at:at + n]
            at += n
        free = np.full(total, -1, np.int32)
        free[:total - at] = ids[at:]
        st["table"], st["free"] = torch.from_numpy(table).cuda(), torch.from_numpy(free).cuda()
        st["free_count"] = ints([total - at])
        st["old"], st["new"] = ints(old), ints(new)
        tokens = sum(max(0, n - o) for o, n in zip(old, new))
        st["max_new"] = tokens + 7  # a step's slot map has a fixed room
        return st
    Hkv, D = case["Hkv"], case["D"]
    if op == "write":
        T = case["T"]
        pages = -(-T // page) + 3
        st["kp"], st["vp"] = randn(pages, page, Hkv, D), randn(pages, page, Hkv, D)
        if case["packed"]:  # views of one projection's output
            qkv = randn(T, 4 * Hkv, D)
            st["k"], st["v"] = qkv[:, 2 * Hkv:3 * Hkv], qkv[:, 3 * Hkv:]
        else:
            st["k"], st["v"] = randn(T, Hkv, D), randn(T, Hkv, D)
        ids = torch.randperm(pages, device="cuda", generator=g)
        t = torch.arange(T, device="cuda")
        slots = ids[t // page] * page + t % page
        st["slots"] = torch.where(t % 1000 == 999, torch.full_like(slots, -1), slots).to(torch.int32)
        return st
    starts, prefix, tails = _shared_lengths(case)
    B = case["B"]
    lens = [0] * B
    rows, used = [[] for _ in range(B)], 1
    for p, P in enumerate(prefix):
        whole = P // page
        common = list(range(used, used + whole))
        used += whole
        for b in range(starts[p], starts[p + 1]):
            lens[b] = P + tails[b]
            more = -(-lens[b] // page) - whole
            rows[b] = common + list(range(used, used + more))
            used += more
    ids = list(range(1, used))
    rng.shuffle(ids)
    ids = [0] + ids
    width = max(len(r) for r in rows)
    st["kp"], st["vp"] = randn(used, page, Hkv, D), randn(used, page, Hkv, D)
    st["table"] = ints([[ids[i] for i in r] + [0] * (width - len(r)) for r in rows])
    for p, P in enumerate(prefix):  # a prefix that ends inside a page: every member has a copy of its end
        r = P % page
        if r:
            for b in range(starts[p] + 1, starts[p + 1]):
                src, dst = ids[rows[starts[p]][P // page]], ids[rows[b][P // page]]
                st["kp"][dst, :r] = st["kp"][src, :r]
                st["vp"][dst, :r] = st["vp"][src, :r]
    st["seqlens"], st["starts"], st["prefix"] = ints(lens), ints(starts), ints(prefix)
    st["host"] = (starts, prefix, lens)  # the scheduler that made the groups knows them
    st["q"] = randn(B, case["Sq"], case["Hq"], D)
    st["scale"] = D ** -0.5
    return st


# ----------------------------------------------------------------------------
# The plain forms
# ----------------------------------------------------------------------------
def _part(q, k, v, scale, ok):
    """Of q [H, R, D] over k, v [H, n, D]: maximum, sum and sum of values."""
    s = (q @ k.transpose(1, 2)).mul_(scale)
    if ok is not None:
        s.masked_fill_(~ok, -math.inf)
    m = s.amax(-1, keepdim=True)
    top = torch.where(m == -math.inf, torch.zeros_like(m), m)
    s.sub_(top).exp_()
    return m, s.sum(-1, keepdim=True), s @ v


def _plain_shared(st):
    c = st["case"]
    Sq, Hq, Hkv, D, page = c["Sq"], c["Hq"], c["Hkv"], c["D"], c["page"]
    G = Hq // Hkv
    starts, prefix, lens = st["host"]
    out = torch.empty_like(st["q"])
    lse = torch.empty(st["q"].shape[:3], device="cuda")

    def keys(b, lo, hi):
        ids = st["table"][b, lo // page:-(-hi // page)].long()
        off = lo - lo // page * page
        return [x[ids].reshape(-1, Hkv, D)[off:off + hi - lo].float().transpose(0, 1)
                for x in (st["kp"], st["vp"])]

    s = torch.arange(Sq, device="cuda").repeat_interleave(G)
    for p, P in enumerate(prefix):
        b0, b1 = starts[p], starts[p + 1]
        n = b1 - b0
        q = st["q"][b0:b1].float().reshape(n, Sq, Hkv, G, D).permute(2, 0, 1, 3, 4).reshape(Hkv, n * Sq * G, D)
        m0, l0, o0 = _part(q, *keys(b0, 0, P), st["scale"], None)
        for b in range(b0, b1):
            r = slice((b - b0) * Sq * G, (b - b0 + 1) * Sq * G)
            L = lens[b]
            ok = torch.arange(P, L, device="cuda") <= (L - Sq + s)[:, None]
            m1, l1, o1 = _part(q[:, r], *keys(b, P, L), st["scale"], ok)
            m = torch.maximum(m0[:, r], m1)
            w0, w1 = torch.exp(m0[:, r] - m), torch.exp(m1 - m)
            l = w0 * l0[:, r] + w1 * l1
            o = (w0 * o0[:, r] + w1 * o1) / l
            out[b] = o.reshape(Hkv, Sq, G, D).transpose(0, 1).reshape(Sq, Hq, D).to(out.dtype)
            lse[b] = (m + torch.log(l)).reshape(Hkv, Sq, G).transpose(0, 1).reshape(Sq, Hq)
    return out, lse


def _plain_sample(st):
    x = st["logits"].float()
    B, V = x.shape
    top = x.amax(-1, keepdim=True).double()
    T = st["temperature"].double()[:, None]
    w = torch.where(T > 0, torch.exp((x.double() - top) / T), (x.double() == top).double())
    s, order = torch.sort(x, dim=-1, descending=True, stable=True)
    ws = torch.gather(w, 1, order)
    rank = torch.arange(V, device="cuda")
    keep = (T > 0) | (rank == 0)
    if st["top_k"] is not None:
        k = st["top_k"][:, None]
        keep = keep & ((rank < k) | (k <= 0))
    if st["top_p"] is not None:
        p = st["top_p"].double()[:, None]
        wk = ws * keep
        c = torch.cumsum(wk, -1)
        keep = keep & ((c - wk < p * c[:, -1:]) | (p >= 1) | (rank == 0))
    if st["min_p"] is not None:
        keep = keep & (ws >= st["min_p"].double()[:, None])
    w = torch.zeros_like(w).scatter_(1, order, ws * keep)
    c = torch.cumsum(w, -1)
    total = c[:, -1:]
    token = (c <= st["u"].double()[:, None] * total).sum(-1).int()
    if st["case"]["probs"]:
        return token, (w / total).float()
    return token


def _plain_pages(st):
    c = st["case"]
    page, max_pages = c["page"], c["max_pages"]
    old, new, table = st["old"].long(), st["new"].long(), st["table"]
    F, cap = st["free_count"].long(), st["free"].numel()
    pages = lambda n: (n + page - 1) // page  # noqa: E731
    j = torch.arange(max_pages, device="cuda")
    gone = (j >= pages(new)[:, None]) & (j < pages(old)[:, None])
    count = torch.cumsum(gone.reshape(-1), 0)
    at = torch.where(gone.reshape(-1), F + count - 1, cap)
    stack = torch.cat([st["free"], st["free"][:1]]).scatter_(0, at, table.reshape(-1))
    have = F + count[-1]
    need = (pages(new) - pages(old)).clamp(min=0)
    tokens = (new - old).clamp(min=0)
    fits = ((torch.cumsum(need, 0) <= have) | (need == 0)) & (torch.cumsum(tokens, 0) <= st["max_new"])
    grow = (tokens > 0) & fits
    lens = torch.where((new < old) | grow, new, old)
    need = need * grow
    before = torch.cumsum(need, 0) - need
    take = (j >= pages(old)[:, None]) & (j < pages(new)[:, None]) & grow[:, None]
    rank = before[:, None] + j - pages(old)[:, None]
    ids = stack[torch.where(take, have - 1 - rank, 0).clamp(min=0)]
    table.copy_(torch.where(take, ids, table))
    left = have - need.sum()
    i = torch.arange(cap, device="cuda")
    st["free"].copy_(torch.where((i >= F) & (i < left), stack[:cap], st["free"]))
    cu = torch.cat([torch.zeros(1, dtype=torch.long, device="cuda"), torch.cumsum(tokens * grow, 0)])
    t = torch.arange(st["max_new"], device="cuda")
    b = (torch.searchsorted(cu, t, right=True) - 1).clamp(max=c["B"] - 1)
    real = t < cu[-1]
    pos = torch.where(real, t - cu[b] + old[b], 0)
    slot = table[b, pos // page].long() * page + pos % page
    slots = torch.where(real, slot, -1).int()
    positions = torch.where(real, pos, 0).int()
    return table, st["free"], lens.int(), left.int(), cu.int(), slots, positions


def _plain_write(st):
    ok = st["slots"] >= 0
    at = st["slots"][ok].long()
    for x, pool in ((st["k"], st["kp"]), (st["v"], st["vp"])):
        pool.view(-1, *pool.shape[2:])[at] = x[ok]
    return st["kp"], st["vp"]


PLAIN = {"shared": _plain_shared, "sample": _plain_sample, "pages": _plain_pages, "write": _plain_write}


def _own(st):
    import attention_fa_fwd_04_gb300 as fa
    op = st["case"]["op"]
    if op == "shared":
        return fa.decode_shared(st["q"], st["kp"], st["vp"], st["table"], st["seqlens"], st["starts"],
                                st["prefix"], st["scale"], lse=True)
    if op == "sample":
        return fa.sample(st["logits"], st["u"], temperature=st["temperature"], top_k=st["top_k"],
                         top_p=st["top_p"], min_p=st["min_p"], probs=True if st["case"]["probs"] else None)
    if op == "pages":
        out = fa.update_pages(st["table"], st["old"], st["new"], st["free"], st["free_count"],
                              st["case"]["page"], st["max_new"])
        return (st["table"], st["free"]) + tuple(out)
    fa.write_pages(st["k"], st["v"], st["kp"], st["vp"], st["slots"])
    return st["kp"], st["vp"]


def run(state):
    return _own(state) if own else PLAIN[state["case"]["op"]](state)


# ----------------------------------------------------------------------------
# From the definitions, in 64 bits
# ----------------------------------------------------------------------------
def _exact_shared(st):
    c = st["case"]
    Sq, Hkv, D, page = c["Sq"], c["Hkv"], c["D"], c["page"]
    G = c["Hq"] // Hkv
    lens = st["seqlens"].tolist()
    outs, lses = [], []
    for b, L in enumerate(lens):  # every sequence by itself, over its own row of the table
        t = torch.arange(L, device="cuda")
        at = st["table"][b].long()[t // page] * page + t % page
        see = t[None] < (L - Sq + 1 + torch.arange(Sq, device="cuda"))[:, None]
        ob, lb = [], []
        for h in range(Hkv):
            k = st["kp"].view(-1, Hkv, D)[at, h].double()
            v = st["vp"].view(-1, Hkv, D)[at, h].double()
            q = st["q"][b, :, h * G:(h + 1) * G].double()
            s = torch.einsum("sgd,nd->sgn", q, k) * st["scale"]
            s = torch.where(see[:, None], s, -math.inf)
            z = torch.logsumexp(s, -1)
            ob.append(torch.exp(s - z[..., None]) @ v)
            lb.append(z)
        outs.append(torch.cat(ob, 1))
        lses.append(torch.cat(lb, 1))
    return torch.stack(outs), torch.stack(lses)


def _exact_sample(st):
    tokens, probs = [], []
    T, u = st["temperature"].tolist(), st["u"].tolist()
    ks, ps, mps = (None if st[n] is None else st[n].tolist() for n in ("top_k", "top_p", "min_p"))
    for b, row in enumerate(st["logits"].float().cpu().numpy().astype(np.float64)):
        order = np.argsort(-row, kind="stable")
        kept = len(order)
        if T[b] > 0:
            z = np.exp((row[order] - row[order[0]]) / T[b])
        else:
            z, kept = np.ones(len(order)), 1
        if ks and ks[b] > 0:
            kept = min(kept, ks[b])
        if ps and ps[b] < 1:
            run_sum = np.concatenate([[0.0], np.cumsum(z[:kept])])
            kept = max(1, int(np.searchsorted(run_sum[:kept], ps[b] * run_sum[kept], side="left")))
        if mps:
            kept = min(kept, max(1, int((z >= mps[b]).sum())))
        chosen = np.sort(order[:kept])
        w = np.exp((row[chosen] - row[order[0]]) / T[b]) if T[b] > 0 else np.ones(1)
        c = np.cumsum(w)
        tokens.append(int(chosen[min(np.searchsorted(c, u[b] * c[-1], side="right"), kept - 1)]))
        if st["case"]["probs"]:
            p = np.zeros(len(row))
            p[chosen] = w / c[-1]
            probs.append(torch.from_numpy(p))
    tokens = torch.tensor(tokens, dtype=torch.int32)
    return (tokens, torch.stack(probs)) if st["case"]["probs"] else tokens


def _exact_pages(st):
    page = st["case"]["page"]
    table, old, new = st["table"].tolist(), st["old"].tolist(), st["new"].tolist()
    before = st["free_count"].item()
    stack, held = st["free"].tolist()[:before], st["free"].tolist()[before:]
    for row, o, n in zip(table, old, new):
        if n < o:
            stack += row[-(-n // page):-(-o // page)]
    lens, cu, slots, positions = [], [0], [], []  # (there is room for all of them)
    for row, o, n in zip(table, old, new):
        for i in range(-(-o // page), -(-n // page)):
            row[i] = stack.pop()
        slots += [row[t // page] * page + t % page for t in range(o, n)]
        positions += list(range(o, n))
        lens.append(n)
        cu.append(len(slots))
    pad = st["max_new"] - len(slots)
    full = stack + held[len(stack) - before:] if len(stack) > before else st["free"].tolist()
    answer = (table, full, lens, [len(stack)], cu, slots + [-1] * pad, positions + [0] * pad)
    return tuple(torch.tensor(x, dtype=torch.int32) for x in answer)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "shared":
        return _exact_shared(st)
    if op == "sample":
        return _exact_sample(st)
    if op == "pages":
        return _exact_pages(st)
    kp, vp = st["kp"].double(), st["vp"].double()
    for t, s in enumerate(st["slots"].tolist()):
        if s >= 0:
            kp[s // case["page"], s % case["page"]] = st["k"][t].double()
            vp[s // case["page"], s % case["page"]] = st["v"][t].double()
    return kp, vp
