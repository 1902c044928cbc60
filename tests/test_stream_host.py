"""Host-side checks of include/kvq_cache.h (no GPU needed, no kernel launched):
exports, workspace sizes, and every refusal before anything reaches the GPU."""
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20                       # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def kb():
    from kv_cache_quantization_kvq_gb300 import build
    build()
    from kv_cache_quantization_kvq_gb300 import binding
    return binding


def test_library_exports_every_declared_symbol(kb):
    with open(os.path.join(ROOT, "include", "kvq_cache.h")) as f:
        declared = set(re.findall(r"KVQ_API\s+[\w\s\*]+?\b(kvq_\w+)\s*\(", f.read()))
    assert declared == set(kb.CACHE_EXPORTS)
    for name in declared:
        assert hasattr(kb.LIB, name), name


def kq(kb, **kw):
    return kb.QParams.asym(**{**dict(bits=4, qmin=0, qmax=15, axis=kb.ALONG_T, group=64, scale_dtype=kb.BF16,
                                     zero_dtype=kb.BF16), **kw})


def vq(kb, **kw):
    return kq(kb, **{**dict(axis=kb.ALONG_C), **kw})


def cache(kb, **kw):
    f = dict(k_codes=FAKE, k_scale=FAKE, k_zero=FAKE, k_resid=FAKE, v_codes=FAKE, v_scale=FAKE, v_zero=FAKE,
             v_resid=FAKE, tq=64, nres=10, resid_rows=64, first=None)
    f.update(kw)
    return kb.kvq_cache(**f)


def attend(kb, q=FAKE, n=1, group=4, kv_heads=2, c=None, k=None, v=None, shape=(4, 128, 128), out=FAKE, lse=FAKE,
           ws=FAKE, ws_B=1 << 40):
    kb.kvq_attend_chunk(q, n, group, kv_heads, c or cache(kb), k or kq(kb), v or vq(kb), shape, out, lse, ws, ws_B, 0)


def weights(kb, q=FAKE, lse=FAKE, n=1, group=4, kv_heads=2, c=None, k=None, shape=(4, 128, 128), sin=None, sout=FAKE,
            stride=200, ws=FAKE, ws_B=1 << 40):
    kb.kvq_attend_weights(q, lse, n, group, kv_heads, c or cache(kb), k or kq(kb), shape, sin, sout, stride, ws, ws_B, 0)


def evict(kb, src=None, dst=None, k=None, v=None, shape=(4, 128, 128), block=64, budget=1, window=0, sin=FAKE, sout=FAKE,
          stride=200, keep=FAKE, ws=FAKE, ws_B=1 << 40):
    kb.kvq_evict_blocks(src or cache(kb, tq=128), dst or cache(kb, tq=128), k or kq(kb), v or vq(kb), shape, block,
                        budget, window, sin, sout, stride, keep, ws, ws_B, 0)


def refused(kb, status, call, *a, **kw):
    with pytest.raises(kb.KvqError) as e:
        call(kb, *a, **kw)
    assert e.value.status == status, str(e.value)


BAD_CACHES = [dict(tq=-1), dict(tq=129), dict(nres=-1), dict(nres=65), dict(resid_rows=-1, nres=0),
              dict(k_codes=None), dict(k_codes=FAKE + 8), dict(k_scale=None), dict(k_scale=FAKE + 2), dict(k_zero=None),
              dict(k_zero=FAKE + 8), dict(k_resid=None), dict(k_resid=FAKE + 4), dict(first=FAKE + 2)]


def test_attend_chunk_refusals(kb):
    for c in BAD_CACHES + [dict(v_codes=None), dict(v_codes=FAKE + 4), dict(v_scale=None), dict(v_scale=FAKE + 1),
                           dict(v_zero=None), dict(v_resid=None), dict(v_resid=FAKE + 2)]:
        refused(kb, kb.EINVAL, attend, c=cache(kb, **c))
    for kw in (dict(q=None), dict(q=FAKE + 2), dict(out=None), dict(out=FAKE + 8), dict(lse=FAKE + 2), dict(n=-1),
               dict(group=0), dict(kv_heads=0), dict(kv_heads=3), dict(shape=(-4, 128, 128)),
               dict(shape=(1 << 40, 1 << 40, 128)), dict(k=kb.QParams(4, 0, -9, 9))):
        refused(kb, kb.EINVAL, attend, **kw)
    for kw in (dict(shape=(4, 128, 96)), dict(shape=(4, 128, 256)), dict(group=65), dict(n=1 << 31),
               dict(k=kq(kb, bits=8)), dict(k=kq(kb, group=16)), dict(k=kq(kb, group=48)), dict(k=kq(kb, group=0)),
               dict(k=kq(kb, axis=kb.ALONG_C)), dict(k=kq(kb, scale_dtype=kb.F32)), dict(k=kq(kb, zero_dtype=kb.I8)),
               dict(v=vq(kb, axis=kb.ALONG_T)), dict(v=vq(kb, group=16)), dict(v=vq(kb, bits=2, qmax=3)),
               dict(v=vq(kb, zero_dtype=kb.F32)), dict(shape=(4, 128, 64), v=vq(kb, group=128))):
        refused(kb, kb.EUNSUPPORTED, attend, **kw)
    big = dict(shape=(4, 1 << 20, 128), c=cache(kb, tq=1 << 20))
    assert kb.kvq_attend_chunk_workspace((4, 1 << 20, 128), 64, 1, 4) > 0
    refused(kb, kb.EWORKSPACE, attend, ws=None, **big)
    refused(kb, kb.EWORKSPACE, attend, ws_B=16, **big)
    refused(kb, kb.EINVAL, attend, ws=FAKE + 16, **big)


def test_attend_weights_refusals(kb):
    for c in BAD_CACHES:
        refused(kb, kb.EINVAL, weights, c=cache(kb, **c))
    for kw in (dict(q=None), dict(lse=None), dict(lse=FAKE + 2), dict(sout=None), dict(sout=FAKE + 2), dict(sin=FAKE + 2),
               dict(stride=73), dict(stride=1 << 60), dict(sin=FAKE + 400), dict(group=0), dict(n=-1), dict(kv_heads=3)):
        refused(kb, kb.EINVAL, weights, **kw)
    for kw in (dict(shape=(4, 128, 32)), dict(k=kq(kb, bits=8)), dict(k=kq(kb, group=40))):
        refused(kb, kb.EUNSUPPORTED, weights, **kw)


def test_evict_blocks_refusals(kb):
    for c in (dict(tq=-64), dict(tq=192), dict(tq=65), dict(tq=128, nres=99), dict(tq=128, k_codes=None),
              dict(tq=128, k_scale=FAKE + 1), dict(tq=128, v_zero=None), dict(tq=128, first=FAKE + 1)):
        refused(kb, kb.EINVAL, evict, src=cache(kb, **c))
    for c in (dict(k_codes=None), dict(v_codes=FAKE + 64), dict(k_zero=FAKE + 2), dict(first=FAKE + 3)):
        refused(kb, kb.EINVAL, evict, dst=cache(kb, **c))
    for kw in (dict(block=0), dict(block=-64), dict(block=96), dict(budget=0), dict(window=-1), dict(window=2),
               dict(sin=None), dict(sout=None), dict(sin=FAKE + 2), dict(sout=FAKE + 4), dict(stride=137), dict(keep=None),
               dict(keep=FAKE + 2), dict(k=kq(kb, group=0)), dict(v=kq(kb, group=48)), dict(shape=(-1, 128, 128))):
        refused(kb, kb.EINVAL, evict, **kw)
    big = dict(shape=(4, 1 << 18, 128), src=cache(kb, tq=1 << 18, nres=0), dst=cache(kb, tq=1 << 18, nres=0), stride=1 << 18,
               sin=FAKE << 4, sout=FAKE << 4)
    want = kb.kvq_evict_blocks_workspace((4, 1 << 18, 128), 64)
    assert want > 0 and kb.kvq_evict_blocks_workspace((4, 128, 128), 64) == 0
    refused(kb, kb.EWORKSPACE, evict, ws=None, **big)
    refused(kb, kb.EWORKSPACE, evict, ws_B=want - 1, **big)
    refused(kb, kb.EINVAL, evict, ws=FAKE + 8, **big)


def test_a_refused_call_leaves_the_counters(kb):
    dst = cache(kb, tq=128, nres=3)
    refused(kb, kb.EINVAL, evict, dst=dst, budget=0)
    assert (dst.tq, dst.nres) == (128, 3)


def test_nothing_to_do_needs_no_buffers(kb):
    none = cache(kb, tq=0, nres=0, **{k: None for k in ("k_codes", "k_scale", "k_zero", "k_resid", "v_codes", "v_scale",
                                                        "v_zero", "v_resid")})
    attend(kb, q=None, out=None, lse=None, n=0, c=none, ws=None, ws_B=0)
    attend(kb, q=None, out=None, lse=None, shape=(0, 128, 128), c=none, ws=None, ws_B=0)
    weights(kb, q=None, lse=None, n=0, c=none, sout=None, ws=None, ws_B=0)
    evict(kb, src=cache(kb, tq=0, nres=0), shape=(0, 128, 128), sin=None, sout=None, keep=None, ws=None, ws_B=0)


def test_workspace_queries_refuse_bad_arguments(kb):
    for call in (kb.kvq_attend_chunk_workspace, kb.kvq_attend_weights_workspace):
        for args in (((4, -1, 128), 0, 1, 1), ((4, 64, 128), -1, 1, 1), ((4, 64, 128), 0, -1, 1), ((4, 64, 128), 0, 1, 0)):
            with pytest.raises(kb.KvqError) as e:
                call(*args)
            assert e.value.status == kb.EINVAL
        with pytest.raises(kb.KvqError) as e:
            call((4, 64, 80), 0, 1, 1)
        assert e.value.status == kb.EUNSUPPORTED
    with pytest.raises(kb.KvqError):
        kb.kvq_evict_blocks_workspace((4, 64, 128), 0)


def test_python_objects_refuse_what_does_not_fit(kb):
    """KVCache and the helpers check sizes, types and devices before any call."""
    import torch
    shape, rows = (2, 128, 128), 64
    ok = {w: tuple(torch.zeros(n, dtype=torch.uint8) for n in kb._store_sizes(shape, q, rows))
          for w, q in (("k", kq(kb)), ("v", vq(kb)))}
    make = dict(shape=shape, kqp=kq(kb), vqp=vq(kb), tq=64, nres=3, resid_rows=rows)
    c = kb.KVCache(**ok, **make)
    assert c.T == 67
    for w in ("k", "v"):
        for i in range(4):
            for bad in (None, torch.zeros(ok[w][i].numel() - 1, dtype=torch.uint8)):
                with pytest.raises(ValueError):
                    kb.KVCache(**{**ok, w: ok[w][:i] + (bad,) + ok[w][i + 1:]}, **make)
    with pytest.raises(ValueError):
        kb.attend_chunk(torch.zeros((1, 1, 8, 128), dtype=torch.bfloat16), c)           # not a CUDA tensor
    for q in (torch.zeros((1, 8, 128), dtype=torch.bfloat16), torch.zeros((3, 1, 8, 128), dtype=torch.bfloat16),
              torch.zeros((2, 1, 8, 64), dtype=torch.bfloat16), torch.zeros((2, 1, 8, 128))):
        with pytest.raises(ValueError):
            kb.attend_chunk(q, c)
    with pytest.raises(ValueError):
        kb.evict_blocks(c, torch.zeros((2, 200)), 1, 0, 64)
    with pytest.raises(ValueError):
        kb.KVCache(**ok, **make, first=torch.zeros(2)).c()
    with pytest.raises(ValueError):
        kb.KVCache(**ok, **make, first=torch.zeros(3, dtype=torch.int32)).c()
