"""What kvq_attend_prompts, kvq_fill_prompts and kvq_attend_shared refuse (no GPU
needed, no kernel launched), and their workspace sizes."""
import pytest

FAKE = 1 << 20                       # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def kb():
    from kv_cache_quantization_kvq_gb300 import build
    build()
    from kv_cache_quantization_kvq_gb300 import binding
    return binding


def kq(kb, **kw):
    return kb.QParams.asym(**{**dict(bits=4, qmin=0, qmax=15, axis=kb.ALONG_T, group=64, scale_dtype=kb.BF16,
                                     zero_dtype=kb.BF16), **kw})


def vq(kb, **kw):
    return kq(kb, **{**dict(axis=kb.ALONG_C), **kw})


def cache(kb, at=FAKE, **kw):
    f = dict.fromkeys(("k_codes", "k_scale", "k_zero", "k_resid", "v_codes", "v_scale", "v_zero", "v_resid"), at)
    return kb.kvq_cache(**{**f, "tq": 64, "nres": 10, "resid_rows": 64, "first": None, **kw})


def refused(kb, status, call, **kw):
    with pytest.raises(kb.KvqError) as e:
        call(kb, **kw)
    assert e.value.status == status, str(e.value)


def prompts(kb, q=FAKE << 8, qs=1024, k=FAKE << 9, ks=256, v=FAKE << 10, vs=256, starts=FAKE, n=3, total=100, group=4,
            heads=2, C=128, out=FAKE << 11, lse=FAKE << 12, ws=FAKE, ws_B=1 << 40):
    kb.kvq_attend_prompts(q, qs, k, ks, v, vs, starts, n, total, group, heads, C, out, lse, ws, ws_B, 0)


def test_attend_prompts_refusals(kb):
    for kw in (dict(q=None), dict(q=(FAKE << 8) + 8), dict(k=None), dict(v=(FAKE << 10) + 2), dict(starts=None),
               dict(starts=FAKE + 2), dict(out=None), dict(out=(FAKE << 11) + 8), dict(lse=(FAKE << 12) + 2), dict(qs=1016),
               dict(qs=1028), dict(ks=128), dict(vs=0), dict(vs=-256), dict(n=-1), dict(total=-1), dict(group=0),
               dict(heads=0), dict(qs=1 << 60)):
        refused(kb, kb.EINVAL, prompts, **kw)
    for kw in (dict(C=96), dict(C=256), dict(group=65, qs=1 << 15), dict(total=1 << 31), dict(n=1 << 31)):
        refused(kb, kb.EUNSUPPORTED, prompts, **kw)
    # out over its inputs: partly over q, in a fused projection's columns, over k or v
    for kw in (dict(out=(FAKE << 8) + 2048), dict(out=FAKE << 8, qs=1536), dict(out=(FAKE << 8) - 4096),
               dict(out=(FAKE << 9) + 16), dict(out=FAKE << 10)):
        refused(kb, kb.EINVAL, prompts, **kw)


def test_attend_prompts_workspace(kb):
    for bad in ((-1, 5, 4, 2, 128), (1, -5, 4, 2, 128), (1, 5, 0, 2, 128), (1, 5, 65, 2, 128), (1, 5, 4, 0, 128),
                (1, 5, 4, 2, 100)):
        with pytest.raises(kb.KvqError):
            kb.kvq_attend_prompts_workspace(*bad)
    assert kb.kvq_attend_prompts_workspace(0, 0, 1, 1, 64) >= 0
    big = kb.kvq_attend_prompts_workspace(64, 1 << 20, 8, 8, 128)
    if big:
        refused(kb, kb.EWORKSPACE, prompts, ws=None)
        refused(kb, kb.EWORKSPACE, prompts, ws_B=1)
        refused(kb, kb.EINVAL, prompts, ws=FAKE + 16)


def fill(kb, k=FAKE << 9, ks=256, v=FAKE << 10, vs=256, starts=FAKE, n=3, total=100, heads=2, c=None, kp=None, vp=None,
         shape=(6, 128, 128)):
    kb.kvq_fill_prompts(k, ks, v, vs, starts, n, total, heads, c or cache(kb, first=FAKE), kp or kq(kb), vp or vq(kb), shape, 0)


def test_fill_prompts_refusals(kb):
    for kw in (dict(k=None), dict(v=None), dict(k=(FAKE << 9) + 8), dict(ks=128), dict(vs=260), dict(starts=None),
               dict(starts=FAKE + 1), dict(n=-1), dict(n=4), dict(total=-1), dict(heads=0), dict(heads=3),
               dict(shape=(5, 128, 128)), dict(c=cache(kb))):
        refused(kb, kb.EINVAL, fill, **kw)
    for c in (dict(tq=-64), dict(tq=192), dict(tq=32), dict(nres=65), dict(nres=-1), dict(k_codes=None), dict(v_codes=FAKE + 8),
              dict(k_scale=None), dict(v_zero=None), dict(k_resid=None), dict(v_resid=FAKE + 2), dict(first=FAKE + 2),
              dict(k_codes=FAKE << 9), dict(v_resid=(FAKE << 10) - 16)):
        refused(kb, kb.EINVAL, fill, c=cache(kb, **{"first": FAKE, **c}))
    for kw in (dict(shape=(6, 128, 96), ks=192, vs=192), dict(kp=kq(kb, bits=8)), dict(kp=kq(kb, group=16)),
               dict(kp=kq(kb, axis=kb.ALONG_C)), dict(vp=vq(kb, axis=kb.ALONG_T)), dict(vp=vq(kb, scale_dtype=kb.F32)),
               dict(vp=vq(kb, bits=2, qmax=3)), dict(total=1 << 31)):
        refused(kb, kb.EUNSUPPORTED, fill, **kw)


def shared(kb, q=FAKE << 8, batch=3, n=1, group=4, heads=2, p=None, kp=None, vp=None, shape=(2, 128, 128), c="own", ckp=None,
           cvp=None, cshape=(6, 128, 128), own_out=None, own_lse=None, out=FAKE << 11, lse=FAKE << 12, ws=FAKE, ws_B=1 << 40):
    c = cache(kb) if c == "own" else c
    kb.kvq_attend_shared(q, batch, n, group, heads, p or cache(kb), kp or kq(kb), vp or vq(kb), shape, c,
                         None if c is None else ckp or kq(kb), None if c is None else cvp or vq(kb),
                         None if c is None else cshape, own_out, own_lse, out, lse, ws, ws_B, 0)


def test_attend_shared_refusals(kb):
    given = dict(c=None, own_out=FAKE << 13, own_lse=FAKE << 14)
    for kw in (dict(q=None), dict(q=(FAKE << 8) + 2), dict(batch=-1), dict(n=-1), dict(group=0), dict(heads=0), dict(heads=1),
               dict(heads=3), dict(batch=4), dict(shape=(1, 128, 128)), dict(shape=(0, 128, 128), heads=0), dict(out=None),
               dict(out=(FAKE << 11) + 8), dict(lse=(FAKE << 12) + 1), dict(out=(FAKE << 8) + 16),
               dict(cshape=(6, 128, 64), cvp=vq(kb, group=64)), dict(p=cache(kb, tq=129)), dict(c=cache(kb, nres=65)),
               dict(p=cache(kb, k_codes=None)), dict(c=cache(kb, v_scale=None)), dict(own_out=FAKE, own_lse=FAKE),
               dict(given, own_lse=None), dict(given, own_out=None), dict(given, own_out=(FAKE << 13) + 2),
               dict(given, own_lse=(FAKE << 14) + 2), dict(given, own_out=(FAKE << 11) + 16),
               dict(given, own_lse=(FAKE << 12) + 4)):
        refused(kb, kb.EINVAL, shared, **kw)
    for kw in (dict(shape=(2, 128, 96)), dict(group=65), dict(batch=1 << 30, cshape=(1 << 31, 0, 128)), dict(kp=kq(kb, bits=8)),
               dict(ckp=kq(kb, group=16)), dict(vp=vq(kb, group=16)), dict(cvp=vq(kb, bits=2, qmax=3))):
        refused(kb, kb.EUNSUPPORTED, shared, **kw)
    want = kb.kvq_attend_shared_workspace((2, 128, 128), 64, (6, 128, 128), 64, 3, 1, 4)
    assert want > 0
    refused(kb, kb.EWORKSPACE, shared, ws=None)
    refused(kb, kb.EWORKSPACE, shared, ws_B=want - 1)
    refused(kb, kb.EINVAL, shared, ws=FAKE + 16)


def test_workspace_covers_every_length(kb):
    """What a call of any tq and nres may need is at most what the query says: larger caches never ask for less."""
    last = 0
    for T in (64, 512, 4096, 65536):
        have = kb.kvq_attend_shared_workspace((8, T, 128), 64, None, 0, 64, 1, 8)
        assert have >= last
        last = have


def test_python_helpers_refuse(kb):
    import torch
    x = torch.zeros((10, 4, 128), dtype=torch.bfloat16)
    st = torch.zeros(2, dtype=torch.int32)
    for bad in ((x, x, x, st), (x.float(), x, x, st), (x[0], x, x, st), (x, x[:, :3], x[:, :3], st), (x, x[:5], x, st)):
        with pytest.raises(ValueError):
            kb.attend_prompts(*bad)
    c = kb.KVCache(*[tuple(torch.zeros(n, dtype=torch.uint8) for n in kb._store_sizes((2, 64, 128), p, 64))
                     for p in (kq(kb), vq(kb))], shape=(2, 64, 128), kqp=kq(kb), vqp=vq(kb), tq=0, nres=0, resid_rows=64,
                   kv_heads=2)
    for bad in ((x, x, st, c, 10), (x[:, :2], x[:, :1], st, c, 10)):
        with pytest.raises(ValueError):
            kb.fill_prompts(*bad)
    with pytest.raises(ValueError):
        kb.attend_shared(x[None], c)
