"""kvq_attend_shared over caches that are shorter than their stores: nothing outside
of the workspace that the query names is written, and the results are those of
a cache as long as its tokens, bit for bit (the splits go by the tokens that
are there)."""
import pytest

from gpu_util import Guarded, kb

pytestmark = pytest.mark.gpu

CAP, G = 8192, 64


@pytest.fixture(scope="module")
def b():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return kb()


def caches(b, outer, heads, tq, nres, C, bits, seed):
    """The same tokens in a store of CAP tokens and in one of tq."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    kw = dict(scale_dtype=b.BF16, zero_dtype=b.BF16)
    kqp, vqp = (b.QParams.asym(bits, 0, 2 ** bits - 1, axis=a, group=G, **kw) for a in (b.ALONG_T, b.ALONG_C))
    x = torch.randn((2, outer, CAP, C), generator=g, device="cuda").bfloat16()
    resid = torch.randn((2, outer, 128, C), generator=g, device="cuda").bfloat16()
    res = []
    for cap in (CAP, tq):
        bufs = []
        for i, p in enumerate((kqp, vqp)):
            store = (None, None, None)
            if cap:
                qt = b.quantize(x[i, :, :cap].contiguous(), p)
                store = (qt.codes, qt.scale, qt.zero)
            bufs.append((*store, resid[i]))
        res.append(b.KVCache(*bufs, shape=(outer, cap, C), kqp=kqp, vqp=vqp, tq=tq, nres=nres, resid_rows=128, kv_heads=heads))
    return res


#  batch, group, n, C, bits, own cache
FORMS = {
    "8 rows": (2, 4, 1, 128, 4, True),
    "16 rows, C 64": (4, 4, 1, 64, 2, True),
    "32 rows": (8, 4, 1, 128, 2, True),
    "32 rows, alone": (8, 4, 1, 128, 4, False),
    "100 rows": (25, 4, 1, 128, 4, True),
    "200 rows, pairs": (25, 8, 1, 128, 4, True),
    "200 rows, C 64": (25, 8, 1, 64, 4, True),
    "600 rows, pairs, two bits": (75, 8, 1, 128, 2, True),
    "600 rows, C 64": (75, 8, 1, 64, 2, True),
    "2100 rows": (75, 4, 7, 128, 4, True),
    "2100 rows, alone": (75, 4, 7, 128, 4, False),
    "chunks": (2, 4, 70, 128, 4, True),
}


@pytest.mark.parametrize("tq", [0, 64, 1088, CAP])
@pytest.mark.parametrize("name", FORMS)
def test_short_caches_in_long_stores(b, name, tq):
    import torch
    B, group, n, C, bits, own = FORMS[name]
    H = 2
    prefix = caches(b, H, H, tq, 70, C, bits, 1)
    short = min(tq, 1088)                        # the requests' own tokens, in stores of CAP too where that is not too much
    mine = caches(b, B * H, H, short, 9, C, bits, 2) if own and B <= 8 else [None, None]
    if own and B > 8:
        one = caches(b, B * H, H, min(short, 64), 9, C, bits, 2)[1]
        mine = [one, one]
    q = torch.randn((B, n, H * group, C), generator=torch.Generator(device="cuda").manual_seed(3), device="cuda").bfloat16()
    got = []
    for p, c in zip(prefix, mine):
        g = Guarded()
        want = b.kvq_attend_shared_workspace(p.shape, p.resid_rows, None if c is None else c.shape, 0 if c is None else c.resid_rows,
                                             B, n, group)
        got.append(b.attend_shared(q, p, c, workspace=g.alloc(want)))
        g.check(f"{name}, {p.shape}")
    for x, y in zip(*got):
        assert torch.equal(x, y) and torch.isfinite(x).all()
    assert b.kvq_wait_timeouts() == 0
