"""What the streaming cache's calls refuse about pairs of caches and buffers (no
GPU needed, no kernel launched)."""
import pytest

FAKE = 1 << 20                       # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def kb():
    from kv_cache_quantization_kvq_gb300 import build
    build()
    from kv_cache_quantization_kvq_gb300 import binding
    return binding


def formats(kb):
    kw = dict(group=64, scale_dtype=kb.BF16, zero_dtype=kb.BF16)
    return [kb.QParams.asym(4, 0, 15, axis=a, **kw) for a in (kb.ALONG_T, kb.ALONG_C)]


def cache(kb, **kw):
    f = dict.fromkeys(("k_codes", "k_scale", "k_zero", "k_resid", "v_codes", "v_scale", "v_zero", "v_resid"), FAKE)
    return kb.kvq_cache(**{**f, "tq": 128, "nres": 10, "resid_rows": 64, "first": None, **kw})


def evict(kb, src, dst, block=64, shape=(4, 128, 128)):
    kb.kvq_evict_blocks(src, dst, *formats(kb), shape, block, 1, 0, FAKE, FAKE, 200, FAKE, FAKE, 1 << 40, 0)


def refused(kb, status, call, *a, **kw):
    with pytest.raises(kb.KvqError) as e:
        call(kb, *a, **kw)
    assert e.value.status == status, str(e.value)


def test_a_destination_that_cannot_hold_the_result(kb):
    """No first for a padded source; fewer buffer rows than tokens in the buffer."""
    for dst in (cache(kb), cache(kb, first=FAKE, resid_rows=9, nres=0)):
        refused(kb, kb.EINVAL, evict, cache(kb, first=FAKE), dst)
        assert dst.tq == 128
    refused(kb, kb.EINVAL, evict, cache(kb), cache(kb, resid_rows=9, nres=0))
    refused(kb, kb.EINVAL, evict, cache(kb, nres=0), cache(kb, resid_rows=-1, nres=0))


def test_a_block_of_more_pieces_than_a_grid_holds(kb):
    """Refused before anything runs: the selection must not have been launched by then."""
    T = 1 << 30
    big = dict(tq=T, nres=0)
    dst = cache(kb, **big)
    with pytest.raises(kb.KvqError) as e:
        kb.kvq_evict_blocks(cache(kb, **big), dst, *formats(kb), (1, T, 128), T, 1, 0, FAKE, FAKE, T, FAKE, FAKE, 1 << 40, 0)
    assert e.value.status == kb.EUNSUPPORTED, str(e.value)
    assert dst.tq == T


def test_outputs_that_overlap_the_queries(kb):
    k, v = formats(kb)

    def attend(kb, out):
        kb.kvq_attend_chunk(FAKE, 2, 4, 2, cache(kb), k, v, (4, 128, 128), out, None, FAKE, 1 << 40, 0)
    for out in (FAKE + 16, FAKE - 16, FAKE + 2 * 2 * 8 * 128 * 2 - 16):
        refused(kb, kb.EINVAL, attend, out)


def test_paddings_that_overlap(kb):
    for at in (FAKE + 4, FAKE - 12):
        refused(kb, kb.EINVAL, evict, cache(kb, first=FAKE), cache(kb, first=at))


def objects(kb, **kw):
    import torch
    shape, rows = (2, 128, 128), 64
    bufs = [tuple(torch.zeros(n, dtype=torch.uint8) for n in kb._store_sizes(shape, q, rows)) for q in formats(kb)]
    return kb.KVCache(*bufs, shape, *formats(kb), **{**dict(tq=64, nres=3, resid_rows=rows, kv_heads=2), **kw})


def test_python_refuses_a_destination_of_other_heads(kb):
    import torch
    with pytest.raises(ValueError, match="dst"):
        kb.evict_blocks(objects(kb), torch.zeros((2, 200)), 1, 0, 64, dst=objects(kb, kv_heads=1))


def test_from_quantized_wants_a_bf16_window(kb):
    """The buffer of a cache is bf16: a float32 window is not one, without a window the codes are all there is."""
    import torch

    def quantized(residual, x_dtype):
        qs = [kb.QParams(p.bits, p.mode, p.qmin, p.qmax, p.axis, p.group, residual, p.scale_dtype, p.zero_dtype)
              for p in formats(kb)]
        return [kb.Quantized(*(torch.zeros(n, dtype=torch.uint8) for n in kb.kvq_quantized_sizes((2, 192, 128), x_dtype, p)[:4]),
                             (2, 192, 128), p, x_dtype) for p in qs]
    assert kb.KVCache.from_quantized(*quantized(64, kb.BF16)).T == 192
    assert kb.KVCache.from_quantized(*quantized(0, kb.F32)).T == 192
    with pytest.raises(ValueError, match="bf16"):
        kb.KVCache.from_quantized(*quantized(64, kb.F32))
    k, v = quantized(64, kb.BF16)[0], quantized(64, kb.F32)[1]
    with pytest.raises(ValueError, match="bf16"):
        kb.KVCache.from_quantized(k, v)
