"""Host-only checks of the draft-tree and norm/rotation entry points: invalid
arguments are refused before anything touches a GPU, empty problems are no-ops."""
import pytest

FAKE = 0x10000  # a 16-byte-aligned non-null address: never dereferenced on these paths


@pytest.fixture(scope="module")
def fa():
    from attention_fa_fwd_04_gb300 import build
    build.build()
    import attention_fa_fwd_04_gb300 as mod
    mod.load()
    return mod


def rope(fa, **kw):
    a = dict(q=FAKE, k=FAKE, qo=FAKE, ko=FAKE, qw=FAKE, kw=FAKE, f=FAKE, pos=FAKE, T=8, Hq=4, Hkv=2,
             D=64, rot=64, qs=256, ks=128, eps=1e-6, il=0, dtype=fa.FA_BF16)
    a.update(kw)
    return fa.fa_qk_norm_rope(*a.values(), 0)


@pytest.mark.parametrize("kw", [
    dict(D=96), dict(rot=8), dict(rot=72), dict(rot=80), dict(rot=0), dict(eps=0.0), dict(eps=-1.0),
    dict(eps=float("nan")), dict(eps=float("inf")), dict(dtype=5), dict(T=-1), dict(Hq=-1),
    dict(T=1 << 31), dict(q=0), dict(q=FAKE + 8), dict(ko=FAKE + 4), dict(qw=FAKE + 2), dict(f=0),
    dict(pos=0), dict(pos=FAKE + 2), dict(qs=255), dict(qs=248), dict(ks=120), dict(ks=-128),
])
def test_rope_rejects(fa, kw):
    assert rope(fa, **kw) == fa.FA_ERR_INVALID_ARG


def test_rope_empty(fa):
    assert rope(fa, T=0, q=0, k=0, f=0) == fa.FA_OK
    assert rope(fa, Hq=0, Hkv=0, q=0, k=0) == fa.FA_OK


def append(fa, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, qo=FAKE, kp=FAKE, vp=FAKE, qw=FAKE, kw=FAKE, f=FAKE, pos=0,
             table=FAKE, lens=FAKE, B=2, N=3, Hq=4, Hkv=2, pages=5, page=32, maxp=4, D=128, rot=128,
             qs=512, ks=256, vs=256, eps=1e-6, il=1, dtype=fa.FA_FP16)
    a.update(kw)
    return fa.fa_qk_norm_rope_append(*a.values(), 0)


@pytest.mark.parametrize("kw", [
    dict(page=16), dict(page=33), dict(page=0), dict(pages=-1), dict(maxp=-1), dict(N=-1), dict(B=-2),
    dict(table=0), dict(lens=0), dict(lens=FAKE + 1), dict(pos=FAKE + 1), dict(kp=FAKE + 8), dict(vp=0),
    dict(v=0), dict(vs=250), dict(vs=248), dict(maxp=1 << 27), dict(D=32), dict(eps=0.0),
    dict(B=1 << 16, N=1 << 16), dict(pages=1 << 30, page=1024),
])
def test_append_rejects(fa, kw):
    assert append(fa, **kw) == fa.FA_ERR_INVALID_ARG


def test_append_empty(fa):
    assert append(fa, B=0, q=0) == fa.FA_OK
    assert append(fa, N=0, q=0) == fa.FA_OK


def backward(fa, **kw):
    a = dict(gq=FAKE, gk=FAKE, q=FAKE, k=FAKE, qw=FAKE, kw=FAKE, f=FAKE, pos=FAKE, dq=FAKE, dk=FAKE,
             dqw=FAKE, dkw=FAKE, T=8, Hq=4, Hkv=2, D=64, rot=32, qs=256, ks=128, eps=1e-6, il=0,
             dtype=fa.FA_BF16)
    a.update(kw)
    return fa.fa_qk_norm_rope_backward(*a.values(), 0)


@pytest.mark.parametrize("kw", [
    dict(dqw=0), dict(dkw=FAKE + 2), dict(dq=0), dict(dk=FAKE + 8), dict(gq=0), dict(gk=FAKE + 4),
    dict(q=0), dict(qs=100), dict(rot=24), dict(eps=0.0), dict(dtype=2), dict(T=-3), dict(pos=0),
    dict(T=0, dqw=0), dict(Hq=0, Hkv=0, dkw=0),
])
def test_backward_rejects(fa, kw):
    assert backward(fa, **kw) == fa.FA_ERR_INVALID_ARG


def tree(fa, **kw):
    a = dict(q=FAKE, kp=FAKE, vp=FAKE, table=FAKE, lens=FAKE, par=FAKE, o=FAKE, lse=0, B=1, N=4, Hq=8,
             Hkv=2, pages=4, page=64, maxp=4, D=128, scale=0.1, dtype=fa.FA_BF16)
    a.update(kw)
    return fa.fa_decode_tree_fwd(*a.values(), 0)


@pytest.mark.parametrize("kw", [
    dict(D=80), dict(dtype=9), dict(scale=float("inf")), dict(scale=float("nan")), dict(page=48),
    dict(page=0), dict(page=-32), dict(Hq=7), dict(Hkv=0), dict(B=-1), dict(N=-1), dict(pages=0),
    dict(pages=-1), dict(maxp=-1), dict(q=0), dict(q=FAKE + 2), dict(o=FAKE + 8), dict(lse=FAKE + 1),
    dict(par=0), dict(par=FAKE + 2), dict(table=0), dict(lens=FAKE + 2), dict(kp=FAKE + 4), dict(vp=0),
    dict(maxp=1 << 26), dict(B=1 << 20, N=64, Hq=64), dict(pages=1 << 30),
    dict(pages=1 << 30, page=1 << 30, maxp=1, Hkv=8),  # (2^71 bytes: a product would wrap to 0)
])
def test_tree_rejects(fa, kw):
    assert tree(fa, **kw) == fa.FA_ERR_INVALID_ARG


def test_tree_limits_and_empty(fa):
    assert tree(fa, N=65) == fa.FA_ERR_UNSUPPORTED
    for kw in (dict(B=0, q=0), dict(N=0, q=0), dict(Hq=0, q=0)):
        assert tree(fa, **kw) == fa.FA_OK


def verify(fa, **kw):
    a = dict(p=FAKE, q=0, tok=FAKE, par=FAKE, u=FAKE, path=FAKE, count=FAKE, nxt=FAKE, B=1, N=4, V=100)
    a.update(kw)
    return fa.fa_verify_tree(*a.values(), 0)


@pytest.mark.parametrize("kw", [
    dict(N=0), dict(N=-1), dict(V=0), dict(V=1 << 30), dict(B=-1), dict(B=1 << 29), dict(p=0),
    dict(p=FAKE + 2), dict(q=FAKE + 1), dict(tok=0), dict(par=0), dict(u=0), dict(path=0), dict(count=0),
    dict(nxt=FAKE + 2),
])
def test_verify_rejects(fa, kw):
    assert verify(fa, **kw) == fa.FA_ERR_INVALID_ARG


def test_verify_limits_and_empty(fa):
    assert verify(fa, N=65) == fa.FA_ERR_UNSUPPORTED
    assert verify(fa, B=0, p=0) == fa.FA_OK


def compact(fa, **kw):
    a = dict(k=FAKE, v=FAKE, table=FAKE, lens=FAKE, path=FAKE, count=FAKE, out=FAKE, layers=2, B=1, N=4,
             Hkv=2, pages=4, page=32, maxp=4, D=64)
    a.update(kw)
    return fa.fa_compact_tree(*a.values(), 0)


@pytest.mark.parametrize("kw", [
    dict(layers=-1), dict(layers=70000), dict(B=-1), dict(B=70000), dict(N=0), dict(Hkv=-1), dict(D=72),
    dict(page=31), dict(pages=-1), dict(maxp=-1), dict(k=0), dict(v=FAKE + 8), dict(table=0),
    dict(lens=0), dict(path=FAKE + 1), dict(count=0), dict(out=0), dict(maxp=1 << 27),
    dict(pages=1 << 30, page=1024),
])
def test_compact_rejects(fa, kw):
    assert compact(fa, **kw) == fa.FA_ERR_INVALID_ARG


def test_compact_limits_and_empty(fa):
    assert compact(fa, N=65) == fa.FA_ERR_UNSUPPORTED
    assert compact(fa, B=0, k=0) == fa.FA_OK


def test_tensor_helpers_refuse(fa):
    """The binding's own checks, on host tensors: shapes and types first, then
    the device."""
    import torch
    i32, bf = torch.int32, torch.bfloat16
    q, kp = torch.zeros(2, 4, 8, 64, dtype=bf), torch.zeros(5, 32, 2, 64, dtype=bf)
    table, lens = torch.zeros(2, 3, dtype=i32), torch.zeros(2, dtype=i32)
    par = torch.zeros(2, 4, dtype=i32)
    good = dict(q=q, kpages=kp, vpages=kp, page_table=table, seqlens=lens, parents=par, scale=0.1)
    for bad, err in ((dict(q=q[0]), ValueError), (dict(q=q.float()), TypeError),
                     (dict(kpages=kp.half()), TypeError), (dict(vpages=kp[:3]), ValueError),
                     (dict(parents=par[:, :3]), ValueError), (dict(parents=par.long()), TypeError),
                     (dict(seqlens=lens[:1]), ValueError), (dict(q=q.transpose(1, 2)), ValueError)):
        with pytest.raises(err):
            fa.decode_tree(**dict(good, **bad))
    with pytest.raises((ValueError, RuntimeError, AssertionError)):  # host tensors
        fa.decode_tree(**good)
    p, u = torch.zeros(2, 4, 10), torch.zeros(2, 4)
    for bad, err in ((dict(target_probs=p[0]), ValueError), (dict(target_probs=p.double()), TypeError),
                     (dict(draft_probs=p[:1]), ValueError), (dict(uniforms=u[:, :2]), ValueError),
                     (dict(uniforms=u.half()), TypeError), (dict(tokens=par.long()), TypeError)):
        with pytest.raises(err):
            fa.verify_tree(**dict(dict(target_probs=p, draft_probs=p, tokens=par, parents=par, uniforms=u),
                                  **bad))
    cnt = torch.zeros(2, dtype=i32)
    for bad, err in ((dict(kpages=kp[0]), ValueError), (dict(vpages=kp.half()), TypeError),
                     (dict(path=par[0]), ValueError), (dict(count=cnt[:1]), ValueError),
                     (dict(kpages=kp.float(), vpages=kp.float()), TypeError)):
        with pytest.raises(err):
            fa.compact_tree(**dict(dict(kpages=kp, vpages=kp, page_table=table, seqlens=lens, path=par,
                                        count=cnt), **bad))
    w, f, pos = torch.ones(64, dtype=bf), torch.ones(32), torch.zeros(2, 4, dtype=i32)
    k = torch.zeros(2, 4, 2, 64, dtype=bf)
    for bad, err in ((dict(k=k[:1]), ValueError), (dict(k=k.half()), TypeError),
                     (dict(q_weight=w[:32]), ValueError), (dict(k_weight=w.float()), TypeError),
                     (dict(inv_freq=f.double()), TypeError), (dict(positions=pos[:, :2]), ValueError),
                     (dict(q=q.transpose(1, 2)), ValueError), (dict(q=q[..., ::2]), ValueError)):
        with pytest.raises(err):
            fa.qk_norm_rope(**dict(dict(q=q, k=k, q_weight=w, k_weight=w, inv_freq=f, positions=pos,
                                        eps=1e-6), **bad))


@pytest.mark.parametrize("shape,stride,ok", [
    ((3, 4, 64), (256, 64, 1), 256), ((3, 4, 64), (512, 64, 1), 512), ((1, 4, 64), (7, 64, 1), 256),
    ((2, 3, 4, 64), (1536, 512, 64, 1), 512), ((2, 3, 4, 64), (2048, 512, 64, 1), None),
    ((2, 1, 4, 64), (512, 9, 64, 1), 512), ((1, 3, 4, 64), (9, 512, 64, 1), 512),
    ((3, 4, 64), (256, 64, 2), None), ((3, 4, 64), (256, 128, 1), None), ((3, 1, 64), (640, 5, 1), 640),
    ((2, 2, 5, 4, 64), (5120, 2560, 512, 64, 1), 512), ((4, 64), (64, 1), 256),
    ((0, 4, 64), (1, 1, 1), 256),
])
def test_token_strides(fa, shape, stride, ok):
    import torch
    t = torch.empty(32768, dtype=torch.float16).as_strided(shape, stride)
    if ok is None:
        with pytest.raises(ValueError):
            fa._token_stride(t)
    else:
        assert fa._token_stride(t) == ok


def test_tree_without_pages_needs_lengths(fa):
    assert tree(fa, maxp=0, pages=0, lens=0) == fa.FA_ERR_INVALID_ARG
    assert tree(fa, maxp=0, pages=0, lens=FAKE + 2) == fa.FA_ERR_INVALID_ARG
