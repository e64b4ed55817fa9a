"""Plain 64-bit forms of the serving-step operators, for the tests: loops that
share no code with the library."""
import numpy as np

from tests.tree_plain import HALF, TINY, U32, f64


# ---------------------------------------------------------------- attention
def decode_paged(q, kp, vp, table, lens, scale):
    """(O, lse, A, E) of new token s over the keys [0, L - Sq + s]: A = sum p |v| / sum p,
    E a bound on the relative error of p from the fp32 scores."""
    q, kp, vp = f64(q), f64(kp), f64(vp)
    B, Sq, Hq, D = q.shape
    page, Hkv = kp.shape[1], kp.shape[2]
    G = Hq // Hkv
    O, A = np.zeros(q.shape), np.zeros(q.shape)
    lse, E = np.full((B, Sq, Hq), -np.inf), np.zeros((B, Sq, Hq))
    for b in range(B):
        L = min(max(int(lens[b]), 0), table.shape[1] * page)
        pos = np.arange(L)
        pid = np.asarray(table[b])[pos // page]
        ok = (pid >= 0) & (pid < kp.shape[0])
        k = kp[np.where(ok, pid, 0), pos % page]
        v = vp[np.where(ok, pid, 0), pos % page]
        for s in range(Sq):
            idx = np.nonzero(ok & (pos <= L - Sq + s))[0]
            if len(idx) == 0:
                continue
            for h in range(Hkv):
                kk, vv, qq = k[idx, h], v[idx, h], q[b, s, h * G:(h + 1) * G]
                sc = qq @ kk.T * scale
                top = sc.max(-1, keepdims=True)
                p = np.exp(sc - top)
                l = p.sum(-1, keepdims=True)
                at = (b, s, slice(h * G, (h + 1) * G))
                O[at] = p @ vv / l
                A[at] = p @ np.abs(vv) / l
                lse[at] = (top + np.log(l))[:, 0]
                E[at] = (D + 4) * U32 * abs(scale) * (np.abs(qq) @ np.abs(kk).T).max(-1)
    return O, lse, A, E


def check_decode(out, lse, q, kp, vp, table, lens, scale):
    """O: P rounded to the inputs' type (relative to A), O rounded once, p off by E + 2^-20
    (scores 2^-24 each; exp2 to 2 fp32 steps, twice where partials are joined; sums) above
    and below the fraction line; fp16 P below 2^-14 is off by 2^-25 of the row's largest."""
    O, ref_lse, A, E = decode_paged(q, kp, vp, table, lens, scale)
    h = HALF[q.dtype]
    p_err = (E + 2.0 ** -20)[..., None]
    vmax = float(np.nan_to_num(np.abs(f64(vp)), nan=0.0, posinf=0.0).max())
    tiny = int(np.max(np.asarray(lens))) * TINY[q.dtype] * vmax
    tol = h * (A + np.abs(O)) * (1 + h) + 2 * p_err * A + tiny + TINY[q.dtype]
    got = f64(out)
    assert np.isfinite(got).all()
    err = np.abs(got - O)
    assert np.all(err <= tol), f"attention off by {np.max(err / np.maximum(tol, 1e-30)):.3g} bounds"
    gl = f64(lse)
    dead = np.isneginf(ref_lse)
    assert np.array_equal(np.isneginf(gl), dead)
    le = np.abs(gl[~dead] - ref_lse[~dead])
    lt = E[~dead] + 2.0 ** -20 + 8 * U32 * np.abs(ref_lse[~dead])
    assert np.all(le <= lt), f"log-sum-exp off by {np.max(le / lt):.3g} bounds"


# ---------------------------------------------------------------- sampling
def sample(row, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """One row: (token, distribution, margin).  margin: how far u and top_p are from where
    the answer changes, in units of the weight."""
    row = np.asarray(row, dtype=np.float64).copy()
    row[np.isnan(row)] = -np.inf
    V = len(row)
    p = np.zeros(V)
    top = row.max()
    if top == -np.inf:
        return -1, p, 1.0
    order = np.lexsort((np.arange(V), -row))
    greedy = not temperature > 0
    with np.errstate(over="ignore", invalid="ignore"):
        w = np.where(row == top, 1.0, 0.0 if greedy or top == np.inf
                     else np.exp((row - top) / min(temperature, 3.4028234663852886e38)))
    w[row == -np.inf] = 0.0
    n, margin = V, 1.0
    if greedy:
        n = 1
    if 0 < top_k < V:
        n = min(n, int(top_k))
    if top_p < 1:
        ws = w[order[:n]]
        before = np.concatenate([[0.0], np.cumsum(ws)[:-1]])
        target = top_p * ws.sum()
        margin = min(margin, np.abs(before[1:] - target).min() / ws.sum() if n > 1 else 1.0)
        n = max(1, int((before < target).sum()))
    if min_p > 0:
        n = min(n, max(1, int((w[order] >= min_p).sum())))
    kept = np.sort(order[:n])
    c = np.cumsum(w[kept])
    aim = max(float(u), 0.0) * c[-1]
    margin = min(margin, np.abs(c[:-1] - aim).min() / c[-1] if n > 1 else 1.0)
    hit = np.nonzero((c > aim) & (w[kept] > 0))[0]
    at = hit[0] if len(hit) else np.nonzero(w[kept] > 0)[0][-1]
    p[kept] = w[kept] / c[-1]
    return int(kept[at]), p, margin


# ---------------------------------------------------------------- page bookkeeping
def update_pages(table, old, new, stack, count, page, max_new, shared=None):
    """Everything one after another on lists: (table, stack, lens, count, cu, slots,
    positions, odd)."""
    table = [list(r) for r in table]
    width, cap = len(table[0]) if table else 0, (len(table[0]) if table else 0) * page
    B = len(old)
    shared = list(shared) if shared is not None else [0] * B
    lens, odd = list(old), False
    pages = lambda n, s: max(-(-n // page), s)  # noqa: E731
    sound = [0 <= o <= cap and 0 <= n <= cap and 0 <= s <= width for o, n, s in zip(old, new, shared)]
    odd = not all(sound)
    back = [(b, j) for b in range(B) if sound[b]
            for j in range(pages(new[b], shared[b]), pages(old[b], shared[b]))]
    held = list(stack)
    if not 0 <= count <= len(stack) or count + len(back) > len(stack):
        return table, held, lens, count, [0] * (B + 1), [-1] * max_new, [0] * max_new, True
    free = held[:count] + [table[b][j] for b, j in back]
    cu, slots, positions = [0], [], []
    need_all = tok_all = 0
    have = len(free)
    for b in range(B):
        if sound[b] and new[b] < old[b]:
            lens[b] = new[b]
        elif sound[b] and new[b] > old[b]:
            want = range(pages(old[b], shared[b]), pages(new[b], shared[b]))
            need_all += len(want)
            tok_all += new[b] - old[b]
            if (need_all <= have or not len(want)) and tok_all <= max_new:
                lens[b] = new[b]
                for j in want:
                    table[b][j] = free.pop()
                for t in range(old[b], new[b]):
                    j, pid = t // page, table[b][t // page]
                    fine = j >= shared[b] and 0 <= pid < (2 ** 31 - 1) // page
                    odd |= j >= shared[b] and not fine
                    slots.append(pid * page + t % page if fine else -1)
                    positions.append(t)
        cu.append(len(slots))
    final = free + held[len(free):] if len(free) > count else held
    pad = max_new - len(slots)
    return table, final, lens, len(free), cu, slots + [-1] * pad, positions + [0] * pad, odd
