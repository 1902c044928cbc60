"""What the Python helpers of serving a batch refuse: calls that are right but for one argument."""
import pytest

from gpu_util import kb

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def b():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return kb()


def empty(b, outer, C=128, rows=128, residual=64):
    import torch
    kw = dict(scale_dtype=b.BF16, zero_dtype=b.BF16, residual=residual)
    kqp, vqp = (b.QParams.asym(4, 0, 15, axis=a, group=64, **kw) for a in (b.ALONG_T, b.ALONG_C))
    bufs = [tuple(torch.zeros(s, dtype=torch.uint8, device="cuda") for s in b._store_sizes((outer, 128, C), p, rows))
            for p in (kqp, vqp)]
    return b.KVCache(*bufs, shape=(outer, 128, C), kqp=kqp, vqp=vqp, tq=0, nres=0, resid_rows=rows, kv_heads=2)


def test_attend_prompts(b):
    import torch
    x = torch.zeros((10, 12, 128), dtype=torch.bfloat16, device="cuda")
    q, k, v = x.split([8, 2, 2], 1)
    st = torch.tensor([0, 10], dtype=torch.int32, device="cuda")
    b.attend_prompts(q, k, v, st)
    wide = torch.zeros((10, 8, 256), dtype=torch.bfloat16, device="cuda")
    for bad in ((q.half(), k, v, st), (q.float(), k, v, st), (q, k.half(), v, st), (q, k, v.float(), st), (q.cpu(), k, v, st),
                (q, k.cpu(), v, st), (q, k, v, st.cpu()), (q, k, v, st.long()), (q, k, v, st[None]), (q, k, v, st[:0]),
                (q, k, v, torch.zeros(4, dtype=torch.int32, device="cuda")[::2]), (q[:9], k, v, st), (q, k[:9], v[:9], st),
                (q, k, v[:, :1], st), (q[:, :7], k, v, st), (q[..., :64], k, v, st), (wide[..., ::2], k, v, st),
                (x[:, ::2][:, :4], k, v, st), (q[0], k, v, st)):
        with pytest.raises(ValueError):
            b.attend_prompts(*bad)
    out, lse = torch.empty((10, 8, 128), dtype=torch.bfloat16, device="cuda"), torch.empty((10, 8), device="cuda")
    b.attend_prompts(q, k, v, st, out, lse)
    for bad in ((out.half(), lse), (out[:9], lse), (x[:, :8], lse), (out.cpu(), lse), (out, lse.half()), (out, lse[:9]),
                (out, lse.T.contiguous().T), (out, lse.cpu())):
        with pytest.raises(ValueError):
            b.attend_prompts(q, k, v, st, *bad)
    both = torch.zeros(10 * 12 * 128, dtype=torch.bfloat16, device="cuda")
    over = both[:10 * 8 * 128].view(10, 8, 128)
    with pytest.raises(b.KvqError):                                       # its last token's rows are the first of k
        b.attend_prompts(q, both[9 * 8 * 128:9 * 8 * 128 + 10 * 2 * 128].view(10, 2, 128), v, st, over)
    with pytest.raises(ValueError):
        b.attend_prompts(q, k, v, st, workspace=torch.empty(1 << 16, dtype=torch.uint8))


def test_fill_prompts(b):
    import torch
    x = torch.zeros((10, 4, 128), dtype=torch.bfloat16, device="cuda")
    k, v = x.split([2, 2], 1)
    st = torch.tensor([0, 10], dtype=torch.int32, device="cuda")
    wide = torch.zeros((10, 2, 256), dtype=torch.bfloat16, device="cuda")
    cache = empty(b, 2)
    for bad in ((k.half(), v, st, 10), (k, v.half(), st, 10), (k.cpu(), v.cpu(), st, 10), (k, v, st.cpu(), 10), (k, v, st.long(), 10),
                (k, v[:9], st, 10), (k[:, :1], v[:, :1], st, 10), (k[..., :64], v[..., :64], st, 10), (k, v, st[:0], 10),
                (wide[..., ::2], wide[..., ::2], st, 10), (k, v, st, -1), (k, v, st, 128 + 128), (k, v, st, 1 << 40)):
        with pytest.raises(ValueError):
            b.fill_prompts(*bad[:3], cache, bad[3])
    with pytest.raises(ValueError):
        b.fill_prompts(k, v, st, empty(b, 2, rows=32), 40)                # the buffer does not hold the residual
    for other in (empty(b, 4), empty(b, 0)):                              # slices for other numbers of prompts
        with pytest.raises(b.KvqError):
            b.fill_prompts(k, v, st, other, 10)
    cache.first = torch.zeros(3, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        b.fill_prompts(k, v, st, cache, 10)
    cache.first = None
    assert (cache.tq, cache.nres) == (0, 0), "a refused call changed the cache"
    b.fill_prompts(k, v, st, cache, 10)
    assert (cache.tq, cache.nres) == (0, 10) and cache.first.tolist() == [0, 0]


def test_attend_shared(b):
    import torch
    prefix, cache = empty(b, 2), empty(b, 6)
    q = torch.zeros((3, 1, 8, 128), dtype=torch.bfloat16, device="cuda")
    b.attend_shared(q, prefix, cache)
    out, lse = b.attend_shared(q, prefix)
    assert out.abs().sum() == 0 and (lse == -float("inf")).all()
    for bad in ((q.half(), prefix, cache), (q.cpu(), prefix, cache), (q[0], prefix, cache), (q[:2], prefix, cache),
                (q[:, :, :7], prefix, cache), (q[..., :64], prefix, cache), (q.transpose(0, 1).expand(3, 3, 8, 128), prefix, cache),
                (q, cache, cache), (q, empty(b, 2, C=64), cache), (q, prefix, empty(b, 6, C=64)), (q, prefix, empty(b, 4))):
        with pytest.raises(ValueError):
            b.attend_shared(*bad)
    for own in ((out, lse.half()), (out.float(), lse), (out[:2], lse), (out, lse[:2]), (out, None), (None, lse), (out.cpu(), lse)):
        with pytest.raises(ValueError):
            b.attend_shared(q, prefix, own=own)
    with pytest.raises(ValueError):
        b.attend_shared(q, prefix, cache, own=(out, lse))
    for kw in (dict(out=out.half()), dict(out=out[:2]), dict(lse=lse.half()), dict(lse=lse[:2]), dict(out=out.cpu())):
        with pytest.raises(ValueError):
            b.attend_shared(q, prefix, cache, **kw)
    with pytest.raises(b.KvqError):
        b.attend_shared(q, prefix, cache, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
