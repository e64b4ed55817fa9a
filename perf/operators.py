"""Cases of the draft-tree decoding operators and of the query/key norm with rotary positions.

Five entry points of the binding are covered:

    qk_norm_rope            RMS norm of every query and key head, then the rotation by position
    qk_norm_rope_backward   its gradient: inputs and both norm weights
    qk_norm_rope_append     the serving form: keys and values go straight into cache pages
    decode_tree             attention of a tree of drafted tokens over a paged cache
    verify_tree             the accepted path of such a tree, and the token after it
    compact_tree            the accepted path's cache rows moved together, new lengths

``run`` computes them with elementary torch operations, or, where ``own`` is
true, through the binding.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
EPS = 1e-6


def listed():
    return [
        # One long prompt at the headline prefill's heads, taken out of a packed qkv projection.
        dict(name="rope_prompt", op="rope", T=8192, Hq=128, Hkv=8, D=128, rot=128, dtype="bf16",
             interleaved=False, theta=500000.0, packed=True),
        # A training step of the MHA prefill's heads.
        dict(name="rope_grad_mha", op="rope_grad", T=16384, Hq=16, Hkv=16, D=128, rot=128,
             dtype="bf16", interleaved=False, theta=10000.0, packed=True),
        # Small ragged fp16 training batch, half of each head rotated, neighbouring pairs.
        dict(name="rope_grad_ragged", op="rope_grad", T=2000, Hq=8, Hkv=8, D=64, rot=32,
             dtype="fp16", interleaved=True, theta=10000.0, packed=False),
        # One new token for each of 16 sequences: latency.
        dict(name="append_token", op="append", B=16, N=1, Hq=8, Hkv=2, D=128, rot=128, dtype="bf16",
             interleaved=False, theta=10000.0, L=65536, page=256),
        # Trees of 64 drafted tokens for 64 sequences.
        dict(name="append_tree", op="append", B=64, N=64, Hq=128, Hkv=8, D=128, rot=128,
             dtype="bf16", interleaved=False, theta=500000.0, L=8192, page=64),
        # One user, a short draft, the single-token decode's heads: latency.
        dict(name="tree_one", op="tree", B=1, N=8, Hq=8, Hkv=2, D=128, dtype="bf16", L=2733,
             page=64),
        # Sixteen users with contexts of different lengths.
        dict(name="tree_batch", op="tree", B=16, N=32, Hq=64, Hkv=8, D=128, dtype="bf16", L=16384,
             page=256),
        # One long context, the largest tree, the headline prefill's heads.
        dict(name="tree_long", op="tree", B=1, N=64, Hq=128, Hkv=8, D=128, dtype="bf16", L=65536,
             page=128),
        # One user, a chain of four greedily drafted tokens after the root: latency.
        dict(name="verify_chain", op="verify", B=1, N=5, V=32000, draft=False, chain=True),
        # Trees of 32 nodes for 64 users, a large vocabulary.
        dict(name="verify_trees", op="verify", B=64, N=32, V=128000, draft=True, chain=False),
        # One user's accepted path in one layer: latency.
        dict(name="compact_one", op="compact", B=1, N=8, keep=4, layers=1, Hkv=2, D=128,
             dtype="bf16", L=2733, page=64),
        # Every layer's caches of 64 users.
        dict(name="compact_layers", op="compact", B=64, N=64, keep=8, layers=24, Hkv=8, D=128,
             dtype="bf16", L=8192, page=64),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "rope_grad", "append", "tree", "tree", "verify", "compact"])
    D = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 5, 8, 16])
    G = rng.choice([1, 2, 3, 4, 7, 8, 16])
    while Hkv * G > 128:
        G = rng.choice([1, 2, 3, 4, 7, 8])
    c = dict(op=op, Hq=Hkv * G, Hkv=Hkv, D=D, dtype=rng.choice(["bf16", "fp16"]))
    rope = dict(rot=rng.choice([16, D // 2, D, D]), interleaved=rng.random() < 0.4,
                theta=rng.choice([10000.0, 500000.0, 1e6]))
    if op in ("rope", "rope_grad"):
        most = 8192 * 136 * 128 // ((c["Hq"] + Hkv) * D * (2 if op == "rope_grad" else 1))
        return dict(c, T=_log(rng, 1, min(65536, most)), packed=rng.random() < 0.5, **rope)
    if op == "append":
        return dict(c, B=_log(rng, 1, 64), N=_log(rng, 1, 64), L=_log(rng, 128, 65536),
                    page=rng.choice([32, 64, 96, 128, 256]), **rope)
    if op == "tree":
        N = _log(rng, 1, 64)
        B = _log(rng, 1, 64)
        most = 65536 * 64 * 128 // (B * max(N * c["Hq"], 512))
        return dict(c, B=B, N=N, L=max(N, _log(rng, 64, max(65, min(65536, most)))),
                    page=rng.choice([32, 64, 96, 128, 256]))
    if op == "verify":
        N = _log(rng, 2, 64)
        V = _log(rng, 1000, 160000)
        B = _log(rng, 1, max(1, min(128, 64 * 32 * 128000 // (N * V))))
        return dict(op=op, B=B, N=N, V=V, draft=rng.random() < 0.6, chain=rng.random() < 0.4)
    N = _log(rng, 2, 64)
    return dict(op=op, B=_log(rng, 1, 64), N=N, keep=rng.randint(1, min(N, 10)),
                layers=rng.choice([1, 2, 7, 24]), Hkv=Hkv, D=D, dtype=c["dtype"],
                L=_log(rng, 128, 8192), page=rng.choice([32, 64, 96, 128]))


def lengths(case):
    """Valid lengths of the sequences, the tree's slots among them: the longest, then others down to a quarter."""
    rng = random.Random("%d %d" % (case["B"], case["L"]))
    L, N = case["L"], case["N"]
    return [max(N, L if b == 0 else rng.randint(max(1, L // 4), L)) for b in range(case["B"])]


def work(case):
    op = case["op"]
    if op in ("rope", "rope_grad"):
        n = case["T"] * (case["Hq"] + case["Hkv"]) * case["D"]
        return {"bytes": n * 2 * (2 if op == "rope" else 3), "flops": n * (8 if op == "rope" else 16)}
    if op == "append":
        t = case["B"] * case["N"] * case["D"]
        return {"bytes": t * (case["Hq"] + 2 * case["Hkv"]) * 4, "flops": t * (case["Hq"] + case["Hkv"]) * 8}
    if op == "tree":
        keys = sum(lengths(case))
        rows = case["B"] * case["N"] * case["Hq"]
        return {"bytes": keys * case["Hkv"] * case["D"] * 4 + rows * (case["D"] * 4 + 4),
                "flops": 4.0 * keys * case["N"] * case["Hq"] * case["D"]}
    if op == "verify":
        rows = case["B"] * case["V"] * (2 if case["draft"] else 1)  # the row where each sequence stops
        return {"bytes": rows * 4, "flops": rows * 2}
    rows = case["B"] * case["layers"] * max(1, case["keep"] - 1)
    return {"bytes": rows * case["Hkv"] * case["D"] * 2 * 2 * 2, "flops": 0}


# ----------------------------------------------------------------------------
# Inputs
# ----------------------------------------------------------------------------
def _tree(B, N, chain, rng):
    """Parents of B trees: node 0 is the root; nodes are numbered level by level, later levels thinner."""
    rows = []
    for _ in range(B):
        p = [-1]
        for s in range(1, N):
            p.append(s - 1 if chain else rng.randint(max(0, (s - 1) // 2 - 2), min(s - 1, max(0, (s - 1) // 2 + 1))))
        rows.append(p)
    return rows


def _depths(parents):
    out = []
    for p in parents:
        d = []
        for s, q in enumerate(p):
            d.append(0 if q < 0 else d[q] + 1)
        out.append(d)
    return out


def _pages(case, lens, g, rng, layers, whole):
    """A page pool and its table. ``whole``: every page of a sequence is its own; else only those under the tree's slots."""
    page, N, Hkv, D = case["page"], case["N"], case["Hkv"], case["D"]
    max_pages = -(-max(lens) // page)
    table = [[0] * max_pages for _ in lens]
    need = [(b, k) for b, L in enumerate(lens)
            for k in range(0 if whole else (L - N) // page, -(-L // page))]
    ids = list(range(1, len(need) + 1))
    rng.shuffle(ids)
    for (b, k), i in zip(need, ids):
        table[b][k] = i
    shape = (len(need) + 1, page, Hkv, D)
    if layers is not None:
        shape = (layers,) + shape
    dt = DTYPES[case["dtype"]]
    k = torch.empty(shape, dtype=dt, device="cuda").normal_(generator=g)
    v = torch.empty(shape, dtype=dt, device="cuda").normal_(generator=g)
    return k, v, torch.tensor(table, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    rng = random.Random(seed)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, st = case["op"], {"case": case}

    def randn(*shape, dtype=None):
        return torch.empty(shape, dtype=dtype or DTYPES[case["dtype"]], device="cuda").normal_(generator=g)

    if op in ("rope", "rope_grad", "append"):
        Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
        st["qw"] = randn(D).mul_(0.2).add_(1)
        st["kw"] = randn(D).mul_(0.2).add_(1)
        i = torch.arange(case["rot"] // 2, dtype=torch.float64, device="cuda")
        st["inv_freq"] = (case["theta"] ** (-2 * i / case["rot"])).float()
    if op in ("rope", "rope_grad"):
        T = case["T"]
        if case["packed"]:  # views of one projection's output
            qkv = randn(T, Hq + 2 * Hkv, D)
            st["q"], st["k"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv]
        else:
            st["q"], st["k"] = randn(T, Hq, D), randn(T, Hkv, D)
        start = rng.randint(0, 1000)
        st["positions"] = torch.arange(start, start + T, dtype=torch.int32, device="cuda")
        if op == "rope_grad":
            st["dq_out"], st["dk_out"] = randn(T, Hq, D), randn(T, Hkv, D)
        return st
    if op == "verify":
        B, N, V = case["B"], case["N"], case["V"]
        parents = _tree(B, N, case["chain"], rng)
        st["parents"] = torch.tensor(parents, dtype=torch.int32, device="cuda")
        logits = randn(B, N, V, dtype=torch.float32).mul_(2.5)
        st["p"] = torch.softmax(logits, -1)
        q = logits.mul_(0.95).add_(torch.empty_like(logits).normal_(generator=g), alpha=0.4)
        q = torch.softmax(q, -1)
        from_row = (torch.arange(B, device="cuda")[:, None] * N + st["parents"].clamp(min=0)).reshape(-1)
        rows = q.reshape(B * N, V)[from_row]
        tokens = torch.multinomial(rows, 1, generator=g).reshape(B, N)
        st["tokens"] = tokens.to(torch.int32)
        st["q"] = q if case["draft"] else None
        st["u"] = torch.rand(B, N, device="cuda", generator=g)
        return st
    lens = lengths(case)
    B, N = case["B"], case["N"]
    st["seqlens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    if op == "compact":
        st["kp"], st["vp"], st["table"] = _pages(case, lens, g, rng, case["layers"], False)
        path = [[0] + sorted(rng.sample(range(1, N), case["keep"] - 1)) for _ in range(B)]
        path = [p + [-1] * (N - len(p)) for p in path]
        st["path"] = torch.tensor(path, dtype=torch.int32, device="cuda")
        st["count"] = torch.full((B,), case["keep"], dtype=torch.int32, device="cuda")
        return st
    st["kp"], st["vp"], st["table"] = _pages(case, lens, g, rng, None, op == "tree")
    parents = _tree(B, N, False, rng)
    if op == "append":
        W = case["Hq"] + 2 * case["Hkv"]
        qkv = randn(B, N, W, case["D"])
        st["q"] = qkv[:, :, :case["Hq"]]
        st["k"] = qkv[:, :, case["Hq"]:case["Hq"] + case["Hkv"]]
        st["v"] = qkv[:, :, case["Hq"] + case["Hkv"]:]
        pos = [[L - N + d for d in ds] for L, ds in zip(lens, _depths(parents))]
        st["positions"] = torch.tensor(pos, dtype=torch.int32, device="cuda")
        return st
    st["q"] = randn(B, N, case["Hq"], case["D"])
    st["parents"] = torch.tensor(parents, dtype=torch.int32, device="cuda")
    st["scale"] = case["D"] ** -0.5
    return st


# ----------------------------------------------------------------------------
# The plain forms
# ----------------------------------------------------------------------------
def _cos_sin(positions, inv_freq):
    a = positions.double()[..., None] * inv_freq.double()
    return torch.cos(a).float()[..., None, :], torch.sin(a).float()[..., None, :]


def _pairs(x, rot, interleaved):
    if interleaved:
        return x[..., 0:rot:2], x[..., 1:rot:2]
    return x[..., :rot // 2], x[..., rot // 2:rot]


def _rotate(x, cos, sin, interleaved):
    rot = 2 * cos.shape[-1]
    a, b = _pairs(x, rot, interleaved)
    y = x.clone()
    ya, yb = _pairs(y, rot, interleaved)
    ra, rb = a * cos - b * sin, b * cos + a * sin
    ya.copy_(ra)
    yb.copy_(rb)
    return y


def _norm(x, w):
    x = x.float()
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()


def _norm_grad(x, w, gy):
    x = x.float()
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    xh = x * r
    gw = gy * w.float()
    dx = r * (gw - xh * (xh * gw).mean(-1, keepdim=True))
    return dx, (gy * xh).double().sum((0, 1)).float()


def _slots(st):
    """Flat token slot in the pool of every tree position [B, N]."""
    page, N = st["case"]["page"], st["case"]["N"]
    slot = st["seqlens"].long()[:, None] - N + torch.arange(N, device="cuda")
    pid = torch.gather(st["table"].long(), 1, slot // page)
    return pid * page + slot % page


def _ancestors(parents):
    """[B, N, N] truth values: node j lies on node s's way to the root (s itself among them)."""
    B, N = parents.shape
    at = torch.arange(N, device=parents.device).expand(B, N)
    nodes = torch.arange(N, device=parents.device)
    p = parents.long()
    see = at[..., None] == nodes
    for _ in range(N - 1):
        at = torch.where(at >= 0, torch.gather(p, 1, at.clamp(min=0)), at)
        see = see | (at[..., None] == nodes)
    return see


def _plain_tree(st):
    c = st["case"]
    B, N, Hq, Hkv, D, page = c["B"], c["N"], c["Hq"], c["Hkv"], c["D"], c["page"]
    G = Hq // Hkv
    see = _ancestors(st["parents"])
    out = torch.empty_like(st["q"])
    lse = torch.empty(B, N, Hq, device="cuda")
    span = st["table"].shape[1] * page
    j = torch.arange(span, device="cuda")
    for b in range(B):
        ids = st["table"][b].long()
        k = st["kp"][ids].reshape(span, Hkv, D).permute(1, 2, 0).float()
        v = st["vp"][ids].reshape(span, Hkv, D).permute(1, 0, 2).float()
        base = st["seqlens"][b].long() - N
        at = (j - base).clamp(0, N - 1)
        ok = (j < base) | ((j < base + N) & see[b][:, at])          # [N, span]
        q = st["q"][b].float().reshape(N, Hkv, G, D).permute(1, 0, 2, 3).reshape(Hkv, N * G, D)
        s = (q @ k).mul_(st["scale"]).reshape(Hkv, N, G, span)
        s.masked_fill_(~ok[:, None, :], -math.inf)
        m = s.amax(-1, keepdim=True)
        s.sub_(m).exp_()
        l = s.sum(-1, keepdim=True)
        o = (s.reshape(Hkv, N * G, span) @ v).reshape(Hkv, N, G, D) / l
        out[b] = o.permute(1, 0, 2, 3).reshape(N, Hq, D).to(out.dtype)
        lse[b] = (m + torch.log(l)).squeeze(-1).permute(1, 0, 2).reshape(N, Hq)
    return out, lse


def _plain_verify(st):
    p, q, tokens, parents, u = st["p"], st["q"], st["tokens"].long(), st["parents"], st["u"]
    B, N, V = p.shape
    dev = p.device
    rows = torch.arange(B, device=dev)
    cur = torch.zeros(B, dtype=torch.long, device=dev)
    path = torch.full((B, N), -1, dtype=torch.int32, device=dev)
    path[:, 0] = 0
    count = torch.ones(B, dtype=torch.long, device=dev)
    r = p[:, 0].double()
    Z = torch.ones(B, dtype=torch.float64, device=dev)
    for s in range(1, N):
        x = tokens[:, s]
        turn = parents[:, s] == cur
        if q is not None:
            qr = q[rows, cur].double()
        else:
            qr = torch.zeros_like(r).scatter_(1, x[:, None], 1.0)
        yes = turn & (u[:, s].double() * qr[rows, x] * Z < r[rows, x])
        no = turn & ~yes
        rest = (r - Z[:, None] * qr).clamp(min=0) if q is not None else r * (1 - qr)
        mass = rest.sum(-1) if q is not None else Z - r[rows, x]
        r = torch.where(no[:, None], rest, torch.where(yes[:, None], p[:, s].double(), r))
        Z = torch.where(no, mass, torch.where(yes, 1.0, Z))
        cur = torch.where(yes, s, cur)
        path[rows, count.clamp(max=N - 1)] = torch.where(yes, s, path[rows, count.clamp(max=N - 1)].long()).int()
        count = count + yes
    c = torch.cumsum(r, -1)
    aim = u[:, 0].double() * c[:, -1]
    nxt = (c <= aim[:, None]).sum(-1)
    return path, count.int(), nxt.int()


def _plain_compact(st):
    c = st["case"]
    N = c["N"]
    slots = _slots(st)
    i = torch.arange(N, device="cuda")
    moved = (i < st["count"][:, None]) & (st["path"] >= 0)
    src = torch.gather(slots, 1, torch.where(moved, st["path"].long(), i)).reshape(-1)
    dst = slots.reshape(-1)
    for pool in (st["kp"], st["vp"]):
        flat = pool.view(c["layers"], -1, c["Hkv"] * c["D"])
        flat[:, dst] = flat[:, src]
    return st["kp"], st["vp"], st["seqlens"] - N + st["count"]


def _plain(st):
    c = st["case"]
    op = c["op"]
    if op == "tree":
        return _plain_tree(st)
    if op == "verify":
        return _plain_verify(st)
    if op == "compact":
        return _plain_compact(st)
    cos, sin = _cos_sin(st["positions"], st["inv_freq"])
    dt = DTYPES[c["dtype"]]
    if op == "rope_grad":
        back = []
        for x, w, g in ((st["q"], st["qw"], st["dq_out"]), (st["k"], st["kw"], st["dk_out"])):
            back.append(_norm_grad(x, w, _rotate(g.float(), cos, -sin, c["interleaved"])))
        return back[0][0].to(dt), back[1][0].to(dt), back[0][1], back[1][1]
    q = _rotate(_norm(st["q"], st["qw"]), cos, sin, c["interleaved"]).to(dt)
    k = _rotate(_norm(st["k"], st["kw"]), cos, sin, c["interleaved"]).to(dt)
    if op == "rope":
        return q, k
    dst = _slots(st).reshape(-1)
    st["kp"].view(-1, c["Hkv"], c["D"])[dst] = k.reshape(-1, c["Hkv"], c["D"])
    st["vp"].view(-1, c["Hkv"], c["D"])[dst] = st["v"].reshape(-1, c["Hkv"], c["D"])
    return q, st["kp"], st["vp"]


def _own(st):
    import attention_fa_fwd_04_gb300 as fa
    c = st["case"]
    op = c["op"]
    if op == "rope":
        return fa.qk_norm_rope(st["q"], st["k"], st["qw"], st["kw"], st["inv_freq"], st["positions"], EPS,
                               interleaved=c["interleaved"])
    if op == "rope_grad":
        return fa.qk_norm_rope_backward(st["dq_out"], st["dk_out"], st["q"], st["k"], st["qw"], st["kw"],
                                        st["inv_freq"], st["positions"], EPS, interleaved=c["interleaved"])
    if op == "append":
        q = fa.qk_norm_rope_append(st["q"], st["k"], st["v"], st["qw"], st["kw"], st["inv_freq"], st["kp"],
                                   st["vp"], st["table"], st["seqlens"], EPS, positions=st["positions"],
                                   interleaved=c["interleaved"])
        return q, st["kp"], st["vp"]
    if op == "tree":
        return fa.decode_tree(st["q"], st["kp"], st["vp"], st["table"], st["seqlens"], st["parents"],
                              st["scale"], lse=True)
    if op == "verify":
        return fa.verify_tree(st["p"], st["q"], st["tokens"], st["parents"], st["u"])
    lens = fa.compact_tree(st["kp"], st["vp"], st["table"], st["seqlens"], st["path"], st["count"])
    return st["kp"], st["vp"], lens


def run(state):
    return _own(state) if own else _plain(state)


# ----------------------------------------------------------------------------
# From the definitions, in 64 bits
# ----------------------------------------------------------------------------
def _turn(x, pos, inv_freq, interleaved, sign):
    """Pairs as complex numbers, times exp(sign i pos f)."""
    rot = 2 * inv_freq.numel()
    head, rest = x[..., :rot], x[..., rot:]
    if interleaved:
        z = torch.view_as_complex(head.unflatten(-1, (-1, 2)).contiguous())
    else:
        z = torch.complex(head[..., :rot // 2].contiguous(), head[..., rot // 2:].contiguous())
    ang = sign * torch.outer(pos.reshape(-1).double(), inv_freq.double()).reshape(*pos.shape, 1, -1)
    z = z * torch.polar(torch.ones_like(ang), ang)
    if interleaved:
        head = torch.view_as_real(z).flatten(-2)
    else:
        head = torch.cat([z.real, z.imag], -1)
    return torch.cat([head, rest], -1)


def _exact_rope(x, w, pos, inv_freq, interleaved):
    x = x.double()
    rms = (torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2 / x.shape[-1] + EPS) ** 0.5
    return _turn(x / rms * w.double(), pos, inv_freq, interleaved, 1.0)


def _exact_rope_grad(x, w, g, pos, inv_freq, interleaved):
    x = x.double()
    D = x.shape[-1]
    gy = _turn(g.double(), pos, inv_freq, interleaved, -1.0)
    rms = ((x * x).sum(-1, keepdim=True) / D + EPS) ** 0.5
    t = gy * w.double()
    dx = t / rms - x * (t * x).sum(-1, keepdim=True) / (D * rms ** 3)
    return dx, torch.einsum("thd,thd->d", gy, x / rms)


def _exact_tree(st):
    c = st["case"]
    N, Hkv, D, page = c["N"], c["Hkv"], c["D"], c["page"]
    G = c["Hq"] // Hkv
    outs, lses = [], []
    parents, lens = st["parents"].tolist(), st["seqlens"].tolist()
    for b, L in enumerate(lens):
        slots = [int(st["table"][b, i]) for i in range(-(-L // page))]
        idx = (torch.tensor(slots, device="cuda")[:, None] * page + torch.arange(page, device="cuda")).reshape(-1)[:L]
        mask = torch.zeros(N, L, dtype=torch.bool)
        mask[:, :L - N] = True
        for s in range(N):
            a = s
            while a >= 0:
                mask[s, L - N + a] = True
                a = parents[b][a]
        mask = mask.cuda()
        ob, lb = [], []
        for h in range(Hkv):
            k = st["kp"].view(-1, Hkv, D)[idx, h].double()
            v = st["vp"].view(-1, Hkv, D)[idx, h].double()
            q = st["q"][b, :, h * G:(h + 1) * G].double()
            oh, lh = [], []
            for i in range(G):
                s = torch.where(mask, (q[:, i] @ k.T) * st["scale"], -math.inf)
                z = torch.logsumexp(s, -1)
                oh.append(torch.exp(s - z[:, None]) @ v)
                lh.append(z)
            ob.append(torch.stack(oh, 1))
            lb.append(torch.stack(lh, 1))
        outs.append(torch.cat(ob, 1))
        lses.append(torch.cat(lb, 1))
    return torch.stack(outs), torch.stack(lses)


def _exact_verify(st):
    B, N, V = st["p"].shape
    tokens, parents, u = st["tokens"].tolist(), st["parents"].tolist(), st["u"].double().tolist()
    paths, counts, nexts = [], [], []
    for b in range(B):
        node, kept = 0, [0]
        while True:
            r, mass, down = st["p"][b, node].double().clone(), 1.0, None
            for s in [s for s in range(1, N) if parents[b][s] == node]:
                x = tokens[b][s]
                if st["q"] is None:
                    if u[b][s] * mass < float(r[x]):
                        down = s
                        break
                    mass -= float(r[x])
                    r[x] = 0.0
                else:
                    d = st["q"][b, node].double()
                    if u[b][s] * float(d[x]) * mass < float(r[x]):
                        down = s
                        break
                    r = torch.relu(r - mass * d)
                    mass = float(r.sum())
            if down is None:
                break
            node = down
            kept.append(node)
        c = r.cumsum(0)
        nexts.append(int(torch.searchsorted(c, c[-1:] * u[b][0], right=True)))
        counts.append(len(kept))
        paths.append(kept + [-1] * (N - len(kept)))
    return tuple(torch.tensor(t, dtype=torch.int32) for t in (paths, counts, nexts))


def exact(case, seed):
    st = prepare(case, seed)
    op, page, N = case["op"], case.get("page"), case.get("N")
    if op == "tree":
        return _exact_tree(st)
    if op == "verify":
        return _exact_verify(st)
    if op == "rope":
        return tuple(_exact_rope(st[x], st[w], st["positions"], st["inv_freq"], case["interleaved"])
                     for x, w in (("q", "qw"), ("k", "kw")))
    if op == "rope_grad":
        a, b = (_exact_rope_grad(st[x], st[w], st[g], st["positions"], st["inv_freq"], case["interleaved"])
                for x, w, g in (("q", "qw", "dq_out"), ("k", "kw", "dk_out")))
        return a[0], b[0], a[1], b[1]
    kp, vp = st["kp"].double(), st["vp"].double()
    table, lens = st["table"].tolist(), st["seqlens"].tolist()

    def where(b, i):
        t = lens[b] - N + i
        return table[b][t // page], t % page

    if op == "append":
        k = _exact_rope(st["k"], st["kw"], st["positions"], st["inv_freq"], case["interleaved"])
        for b in range(case["B"]):
            for i in range(N):
                pid, at = where(b, i)
                kp[pid, at], vp[pid, at] = k[b, i], st["v"][b, i].double()
        return _exact_rope(st["q"], st["qw"], st["positions"], st["inv_freq"], case["interleaved"]), kp, vp
    path, count = st["path"].tolist(), st["count"].tolist()
    for b in range(case["B"]):
        for i in range(count[b]):
            (p0, a0), (p1, a1) = where(b, path[b][i]), where(b, i)
            kp[:, p1, a1], vp[:, p1, a1] = kp[:, p0, a0].clone(), vp[:, p0, a0].clone()
    return kp, vp, torch.tensor([L - N + n for L, n in zip(lens, count)], dtype=torch.int32)
