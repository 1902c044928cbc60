"""A batch without requests through the Python helpers."""
import pytest

from gpu_util import kb

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def b():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return kb()


@pytest.mark.parametrize("total", [0, 7])
@pytest.mark.parametrize("tokens", [0, 150])
def test_no_requests(b, total, tokens):
    import torch
    kw = dict(scale_dtype=b.BF16, zero_dtype=b.BF16, residual=64)
    kqp, vqp = (b.QParams.asym(4, 0, 15, axis=a, group=64, **kw) for a in (b.ALONG_T, b.ALONG_C))
    none = torch.empty(0, dtype=torch.uint8, device="cuda")
    cache = b.KVCache((none,) * 4, (none,) * 4, shape=(0, 128, 128), kqp=kqp, vqp=vqp, tq=0, nres=0, resid_rows=128, kv_heads=2)
    starts = torch.zeros(1, dtype=torch.int32, device="cuda")
    x = torch.randn((total, 12, 128), device="cuda").bfloat16()
    q, k, v = x.split([8, 2, 2], 1)
    out, lse = b.attend_prompts(q, k, v, starts)
    assert out.shape == (total, 8, 128) and lse.shape == (total, 8)
    b.fill_prompts(k, v, starts, cache, tokens)
    assert (cache.tq, cache.nres) == ((0, 0) if tokens == 0 else (64, 86)) and cache.first.numel() == 0
    sizes = [b._store_sizes((2, 128, 128), p, 128) for p in (kqp, vqp)]
    prefix = b.KVCache(*[tuple(torch.zeros(s, dtype=torch.uint8, device="cuda") for s in z) for z in sizes], shape=(2, 128, 128),
                       kqp=kqp, vqp=vqp, tq=64, nres=10, resid_rows=128, kv_heads=2)
    out, lse = b.attend_shared(torch.empty((0, 1, 8, 128), dtype=torch.bfloat16, device="cuda"), prefix, cache)
    assert out.shape == (0, 1, 8, 128) and lse.shape == (0, 1, 8)
