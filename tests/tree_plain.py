"""Plain 64-bit forms of the draft-tree operators and of the norm with rotary
positions, for the tests: numpy loops that share no code with the library.

Rounding bounds: HALF[dtype] is the largest relative error of one rounding to
that type, U32 the same of fp32.
"""
import numpy as np
import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25}  # half a step below the normal range
U32 = 2.0 ** -24


def f64(t):
    return t.detach().cpu().double().numpy()


# ---------------------------------------------------------------- norm and rotation
def pairs(D, rot, interleaved):
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def angles(positions, inv_freq):
    return np.asarray(positions, dtype=np.float64)[..., None] * f64(inv_freq)


def turn(x, ang, interleaved, sign=1.0):
    a, b = pairs(x.shape[-1], 2 * ang.shape[-1], interleaved)
    c, s = np.cos(ang)[..., None, :], sign * np.sin(ang)[..., None, :]
    y = x.copy()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def pair_size(x, rot, interleaved):
    """|first| + |second| of each element's pair (its own size past rot)."""
    a, b = pairs(x.shape[-1], rot, interleaved)
    y = np.abs(x)
    y[..., a] = y[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
    return y


def norm_rope(x, w, ang, eps, interleaved):
    x = f64(x)
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * f64(w)
    return turn(y, ang, interleaved), pair_size(y, 2 * ang.shape[-1], interleaved)


def check_rope(got, x, w, ang, eps, interleaved):
    """Error of one output: a rounding to its type, and 32 fp32 roundings of the
    pair: about 20 in the sum of squares (16 products in a lane, 3 additions
    across lanes; halved by the root), 4 in the reciprocal root, 2 in the
    scaling, 8 in cosine, sine and their argument, 3 in the turn."""
    ref, size = norm_rope(x, w, ang, eps, interleaved)
    h = HALF[x.dtype]
    tol = h * np.abs(ref) + (1 + h) * 32 * U32 * size + TINY[x.dtype]
    err = np.abs(f64(got) - ref)
    assert np.all(err <= tol), f"norm and rotation off by {np.max(err / tol):.3g} bounds"


def norm_rope_grad(x, w, g, ang, eps, interleaved):
    """dx, dw and the sizes that their rounding errors scale with."""
    x, w, g = f64(x), f64(w), f64(g)
    D = x.shape[-1]
    rot = 2 * ang.shape[-1]
    gy = turn(g, ang, interleaved, -1.0)
    gs = pair_size(g, rot, interleaved)
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    dx = r * (w * gy - x * r * r * (x * w * gy).mean(-1, keepdims=True))
    size = r * (np.abs(w) * gs + np.abs(x) * r * r * (np.abs(x * w) * gs).mean(-1, keepdims=True))
    axes = tuple(range(x.ndim - 1))
    return dx, (gy * x * r).sum(axes), size, (gs * np.abs(x) * r).sum(axes)


def lane_additions(T, Hq, Hkv, D, sms):
    """At most how many rows one lane of the gradient adds up: two blocks of 8
    warps per SM share the rows of both parts by their cost, 256 / D rows of a
    warp side by side and a token's last group filled up; four times an even
    share, and 16 more for what the shares' rounding leaves."""
    at_once = 256 // D
    groups = T * (-(-Hq // at_once) + -(-Hkv // at_once))
    return 4 * -(-groups // (2 * sms * 8)) + 16


def check_weight_grad(got, x, w, g, ang, eps, interleaved, adds):
    """A weight's gradient: 40 fp32 roundings of each product, the additions of a
    lane (adds), and 40 of a warp, a block and the blocks."""
    _, ref, _, size = norm_rope_grad(x, w, g, ang, eps, interleaved)
    tol = (40 + adds + 40) * U32 * size
    err = np.abs(f64(got) - ref)
    assert np.all(err <= tol), f"weight gradient off by {np.max(err / np.maximum(tol, 1e-30)):.3g} bounds"


# ---------------------------------------------------------------- tree attention
def tree_sees(parents, N):
    """see[s][a]: node a lies on node s's way up; usable[s]."""
    see = np.zeros((N, N), bool)
    usable = np.ones(N, bool)
    for s in range(N):
        a, seen = s, []
        while a >= 0:
            seen.append(a)
            p = int(parents[a])
            a = p if -2 <= p < a else -2
        usable[s] = a == -1
        if usable[s]:
            see[s, seen] = True
    return see, usable


def decode_tree(q, kp, vp, table, lens, parents, scale):
    """(O, lse, A, E): A = sum p |v| / sum p, E a bound on the relative error of
    p from the fp32 scores."""
    q, kp, vp = f64(q), f64(kp), f64(vp)
    B, N, Hq, D = q.shape
    page, Hkv = kp.shape[1], kp.shape[2]
    G = Hq // Hkv
    O, A = np.zeros(q.shape), np.zeros(q.shape)
    lse, E = np.full((B, N, Hq), -np.inf), np.zeros((B, N, Hq))
    for b in range(B):
        L = int(lens[b])
        if L < N or L > table.shape[1] * page:
            continue
        see, usable = tree_sees(parents[b], N)
        pos = np.arange(L)
        pid = np.asarray(table[b])[pos // page]
        ok = (pid >= 0) & (pid < kp.shape[0])
        k = kp[np.where(ok, pid, 0), pos % page]
        v = vp[np.where(ok, pid, 0), pos % page]
        for s in range(N):
            if not usable[s]:
                continue
            m = ok.copy()
            m[L - N:] &= see[s]
            idx = np.nonzero(m)[0]
            if len(idx) == 0:
                continue
            for h in range(Hq):
                kk, vv, qq = k[idx, h // G], v[idx, h // G], q[b, s, h]
                sc = kk @ qq * scale
                top = sc.max()
                p = np.exp(sc - top)
                l = p.sum()
                O[b, s, h] = p @ vv / l
                A[b, s, h] = p @ np.abs(vv) / l
                lse[b, s, h] = top + np.log(l)
                E[b, s, h] = (D + 4) * U32 * abs(scale) * (np.abs(kk) @ np.abs(qq)).max()
    return O, lse, A, E


def check_tree(out, lse, q, kp, vp, table, lens, parents, scale):
    """O: P rounded to the inputs' type (relative to A), O rounded once, p off
    by E + 2^-21 (scores; exp2 to 2 fp32 steps; sums) above and below the
    fraction line; fp16 P below 2^-14 is off by 2^-25 of the row's largest."""
    O, ref_lse, A, E = decode_tree(q, kp, vp, table, lens, parents, scale)
    h = HALF[q.dtype]
    p_err = (E + 2.0 ** -21)[..., None]
    vmax = float(np.nan_to_num(np.abs(f64(vp)), nan=0.0, posinf=0.0).max())
    tiny = int(np.max(np.asarray(lens))) * TINY[q.dtype] * vmax
    tol = h * (A + np.abs(O)) * (1 + h) + 2 * p_err * A + tiny + TINY[q.dtype]
    got = f64(out)
    assert np.isfinite(got).all()
    err = np.abs(got - O)
    assert np.all(err <= tol), f"tree attention off by {np.max(err / np.maximum(tol, 1e-30)):.3g} bounds"
    if lse is not None:
        gl = f64(lse)
        dead = np.isneginf(ref_lse)
        assert np.array_equal(np.isneginf(gl), dead)
        le = np.abs(gl[~dead] - ref_lse[~dead])
        lt = E[~dead] + 2.0 ** -20 + 8 * U32 * np.abs(ref_lse[~dead])
        assert np.all(le <= lt), f"log-sum-exp off by {np.max(le / lt):.3g} bounds"


# ---------------------------------------------------------------- verification
def verify(p, q, tokens, parents, u):
    """One sequence: (path, next token)."""
    def clean(x):
        x = np.asarray(x, dtype=np.float64).copy()
        x[~(np.isfinite(x) & (x > 0))] = 0.0
        return x

    N, V = p.shape
    node, path = 0, [0]
    while True:
        r, Z, down = clean(p[node]), 1.0, None
        for c in range(1, N):
            x = int(tokens[c])
            if int(parents[c]) != node or not 0 <= x < V:
                continue
            qr = clean(q[node]) if q is not None else None
            qx = qr[x] if q is not None else 1.0
            if float(u[c]) * qx * Z < r[x]:
                down = c
                break
            if q is not None:
                r = np.maximum(r - Z * qr, 0.0)
                Z = r.sum()
            else:
                Z -= r[x]
                r[x] = 0.0
        if down is None:
            break
        node = down
        path.append(node)
    if not r.sum() > 0:
        r = clean(p[node])
    if not r.sum() > 0:
        return path, -1
    c = np.cumsum(r)
    hit = np.nonzero((c > float(u[0]) * c[-1]) & (r > 0))[0]
    return path, int(hit[0]) if len(hit) else int(np.nonzero(r > 0)[0][-1])


# ---------------------------------------------------------------- compaction
def compact(pool, table, lens, path, count, N):
    """pool [layers, pages, page, ...] moved in place; the new lengths."""
    page = pool.shape[2]
    out = []
    for b, L in enumerate(lens):
        L, n = int(L), int(count[b])
        way = [int(x) for x in path[b][:max(n, 0)]]
        slots = [L - N + i for i in range(N)] if L >= N else []
        cap = table.shape[1] * page
        fine = (0 <= n <= N and L <= cap and all(0 <= x < N for x in way)
                and all(a < c for a, c in zip(way, way[1:])))
        if L < N or not fine:
            out.append(L)
            continue
        moves = [(slots[x], slots[i]) for i, x in enumerate(way) if x != i]
        ids = [int(table[b][s // page]) for m in moves for s in m]
        if any(i < 0 or i >= pool.shape[1] for i in ids):
            out.append(L)
            continue
        for a, c in moves:
            pool[:, int(table[b][c // page]), c % page] = pool[:, int(table[b][a // page]), a % page]
        out.append(L - N + n)
    return out


def random_parents(B, N, rng, unused=0.0):
    rows = []
    for _ in range(B):
        p = [-1]
        for s in range(1, N):
            p.append(-2 if rng.random() < unused else rng.randint(max(0, s // 2 - 2), s - 1))
        rows.append(p)
    return rows
