"""Host-only checks of the serving-step entry points: invalid arguments are refused
before anything touches a GPU, empty problems are no-ops."""
import pytest

FAKE = 0x10000  # a 16-byte-aligned non-null address: never dereferenced on these paths


@pytest.fixture(scope="module")
def fa():
    from attention_fa_fwd_04_gb300 import build
    build.build()
    import attention_fa_fwd_04_gb300 as mod
    mod.load()
    return mod


def shared(fa, **kw):
    a = dict(q=FAKE, kp=FAKE, vp=FAKE, table=FAKE, lens=FAKE, starts=FAKE, prefix=FAKE, o=FAKE, lse=0, B=4,
             Sq=2, Hq=8, Hkv=2, pages=4, page=64, maxp=4, groups=1, D=128, scale=0.1, dtype=fa.FA_BF16)
    a.update(kw)
    return fa.fa_decode_shared_fwd(*a.values(), 0)


@pytest.mark.parametrize("kw", [
    dict(D=80), dict(dtype=2), dict(dtype=9), dict(scale=float("inf")), dict(scale=float("nan")),
    dict(page=48), dict(page=0), dict(page=-32), dict(Hq=7), dict(Hkv=0), dict(B=-1), dict(Sq=-1),
    dict(groups=-1), dict(pages=0), dict(pages=-1), dict(maxp=-1), dict(q=0), dict(q=FAKE + 2),
    dict(o=FAKE + 8), dict(lse=FAKE + 1), dict(starts=0), dict(prefix=0), dict(starts=FAKE + 2),
    dict(prefix=FAKE + 1), dict(table=0), dict(lens=0), dict(lens=FAKE + 2), dict(kp=FAKE + 4), dict(vp=0),
    dict(maxp=1 << 26), dict(B=1 << 20, Sq=64, Hq=64), dict(pages=1 << 30),
    dict(pages=1 << 30, page=1 << 30, maxp=1, Hkv=8),
])
def test_shared_rejects(fa, kw):
    assert shared(fa, **kw) == fa.FA_ERR_INVALID_ARG


def test_shared_limits_and_empty(fa):
    assert shared(fa, groups=1025) == fa.FA_ERR_UNSUPPORTED
    for kw in (dict(B=0, q=0), dict(Sq=0, q=0), dict(Hq=0, q=0)):
        assert shared(fa, **kw) == fa.FA_OK


@pytest.mark.parametrize("kw", [
    dict(B=4_100_000, Sq=17, Hq=1, Hkv=1), dict(B=2_050_000, Sq=17, Hq=2, Hkv=2, groups=0),
    dict(B=8_200_000, Sq=17, Hq=1, Hkv=1, D=64, groups=0), dict(B=1_000_000, Sq=16, Hq=16, Hkv=16, groups=0),
    dict(B=1 << 20, Sq=16, Hq=64, Hkv=8, groups=1024),
])
def test_shared_refuses_partials_past_the_merges_index(fa, kw):
    """More than 2^32 pieces of 16 bytes: rows in two parts of a slot, streamed rows, groups' rows."""
    assert shared(fa, **kw) == fa.FA_ERR_UNSUPPORTED


def sample(fa, **kw):
    a = dict(x=FAKE, u=FAKE, T=0, k=0, p=0, m=0, tok=FAKE, probs=0, rows=3, V=1000, stride=1000,
             dtype=fa.FA_FP32)
    a.update(kw)
    return fa.fa_sample(*a.values(), 0)


@pytest.mark.parametrize("kw", [
    dict(rows=-1), dict(rows=1 << 29), dict(V=0), dict(V=-5), dict(stride=999), dict(dtype=3), dict(x=0),
    dict(x=FAKE + 2), dict(dtype=0, x=FAKE + 1), dict(u=0), dict(u=FAKE + 2), dict(tok=0), dict(T=FAKE + 1),
    dict(k=FAKE + 2), dict(p=FAKE + 3), dict(m=FAKE + 1), dict(probs=FAKE + 2),
])
def test_sample_rejects(fa, kw):
    assert sample(fa, **kw) == fa.FA_ERR_INVALID_ARG


def test_sample_limits_and_empty(fa):
    assert sample(fa, V=1 << 22, stride=1 << 22) == fa.FA_ERR_UNSUPPORTED
    assert sample(fa, V=1 << 20, stride=1 << 20, dtype=fa.FA_BF16) == fa.FA_ERR_UNSUPPORTED
    assert sample(fa, rows=0, x=0) == fa.FA_OK


def update(fa, **kw):
    a = dict(table=FAKE, old=FAKE, new=FAKE, shared=0, pages=FAKE, count=FAKE, lens=FAKE, left=FAKE, cu=FAKE,
             slots=FAKE, pos=FAKE, B=3, page=64, maxp=8, maxf=20, maxn=30)
    a.update(kw)
    return fa.fa_update_pages(*a.values(), 0)


@pytest.mark.parametrize("kw", [
    dict(B=-1), dict(page=16), dict(page=33), dict(page=0), dict(maxp=-1), dict(maxf=-1), dict(maxn=-1),
    dict(maxp=1 << 26), dict(table=0), dict(old=0), dict(new=FAKE + 1), dict(shared=FAKE + 2), dict(pages=0),
    dict(count=0), dict(lens=0), dict(left=FAKE + 2), dict(cu=0), dict(slots=0), dict(pos=FAKE + 1),
])
def test_update_rejects(fa, kw):
    assert update(fa, **kw) == fa.FA_ERR_INVALID_ARG


def test_update_limit(fa):
    assert update(fa, B=4097) == fa.FA_ERR_UNSUPPORTED


def write(fa, **kw):
    a = dict(k=FAKE, v=FAKE, kp=FAKE, vp=FAKE, slots=FAKE, T=9, Hkv=2, pages=4, page=32, D=64, ks=128, vs=256)
    a.update(kw)
    return fa.fa_write_pages(*a.values(), 0)


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(T=1 << 31), dict(Hkv=-1), dict(pages=-1), dict(D=96), dict(page=40), dict(page=0),
    dict(k=0), dict(k=FAKE + 8), dict(v=FAKE + 2), dict(kp=0), dict(vp=FAKE + 4), dict(slots=0),
    dict(slots=FAKE + 2), dict(ks=120), dict(ks=132), dict(vs=-256), dict(pages=1 << 26, page=32),
])
def test_write_rejects(fa, kw):
    assert write(fa, **kw) == fa.FA_ERR_INVALID_ARG


def test_write_empty(fa):
    assert write(fa, T=0, k=0) == fa.FA_OK
    assert write(fa, Hkv=0, k=0) == fa.FA_OK


def test_tensor_helpers_refuse(fa):
    """The binding's own checks, on host tensors: shapes and types first, then the device."""
    import torch
    i32, bf = torch.int32, torch.bfloat16
    q, kp = torch.zeros(2, 4, 8, 64, dtype=bf), torch.zeros(5, 32, 2, 64, dtype=bf)
    table, lens, g1 = torch.zeros(2, 3, dtype=i32), torch.zeros(2, dtype=i32), torch.zeros(1, dtype=i32)

    def refuses(call, good, cases):
        for bad, err in cases:
            with pytest.raises(err):
                call(**dict(good, **bad))
        with pytest.raises(ValueError, match="CUDA"):
            call(**good)

    refuses(fa.decode_shared,
            dict(q=q, kpages=kp, vpages=kp, page_table=table, seqlens=lens, group_starts=lens, prefix_lens=g1,
                 scale=0.1),
            [(dict(q=q[0, 0]), ValueError), (dict(q=q.float()), TypeError), (dict(kpages=kp.half()), TypeError),
             (dict(vpages=kp[:3]), ValueError), (dict(group_starts=g1), ValueError),
             (dict(prefix_lens=lens), ValueError), (dict(prefix_lens=g1.float()), TypeError),
             (dict(seqlens=lens[:1]), ValueError), (dict(q=q.transpose(1, 2)), ValueError),
             (dict(group_starts=[0, 2]), TypeError)])
    x, u = torch.zeros(3, 50), torch.zeros(3)
    refuses(fa.sample, dict(logits=x, uniforms=u),
            [(dict(logits=x.double()), TypeError), (dict(logits=x.t()), ValueError),
             (dict(logits=x[:, :0]), ValueError), (dict(logits=x[:1].expand(3, 50)), ValueError)])
    refuses(fa.update_pages,
            dict(page_table=table, old_lens=lens, new_lens=lens, free_pages=g1, free_count=g1, page_size=32,
                 max_new=4),
            [(dict(page_table=table.long()), TypeError), (dict(page_table=lens), ValueError),
             (dict(new_lens=g1), ValueError), (dict(free_count=lens), ValueError),
             (dict(free_pages=table), ValueError), (dict(max_new=-1), ValueError), (dict(max_new=1.5), TypeError),
             (dict(page_size=1 << 40), ValueError), (dict(shared_pages=g1), ValueError),
             (dict(page_table=table.t().contiguous().t()), ValueError)])
    k = torch.zeros(7, 2, 64, dtype=bf)
    refuses(fa.write_pages, dict(k=k, v=k, kpages=kp, vpages=kp, slots=torch.zeros(7, dtype=i32)),
            [(dict(v=k[:6]), ValueError), (dict(v=k.half()), TypeError), (dict(kpages=kp.half()), TypeError),
             (dict(vpages=kp[:2]), ValueError), (dict(k=k[:, :1], v=k[:, :1]), ValueError),
             (dict(slots=torch.zeros(6, dtype=i32)), ValueError), (dict(slots=torch.zeros(7)), TypeError),
             (dict(k=k.transpose(1, 2), v=k.transpose(1, 2)), ValueError), (dict(kpages=kp[0]), ValueError)])
