"""kvq_evict_blocks between two caches: what an out-of-place call leaves alone, and
caches that share some of their buffers; and shapes at the edge of the launch."""
import numpy as np
import pytest

import stream_util as S
from gpu_util import kb

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def b():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return kb()


def setup(b, seed, first=None, cases=(3, 128, 64 * 12, 64 * 12 + 40, 30, 64)):
    import torch
    rng = np.random.default_rng(seed)
    hc = S.HostCache(rng, *cases, *S.formats())
    sc = np.exp(2 * rng.standard_normal((cases[0], hc.T + 7))).astype(np.float32)
    return hc, sc, hc.device(b, 1, first), torch.from_numpy(sc).cuda()


def test_out_of_place_leaves_the_source(b):
    """dst without scores_out and without first: both are made, nothing of the source changes."""
    import torch
    first = [0, 70, 800]
    hc, sc, cache, ds = setup(b, 1, first)
    dst = hc.device(b)
    assert dst.first is None
    before = [t.clone() for t in (*cache.k, *cache.v, cache.first)]
    got, out, keep = b.evict_blocks(cache, ds, 5, 2, 64, dst=dst)
    assert got is dst and out is not ds and np.array_equal(ds.cpu().numpy(), sc)
    assert all(torch.equal(x, y) for x, y in zip(before, (*cache.k, *cache.v, cache.first)))
    assert (cache.tq, cache.nres, dst.tq, dst.nres) == (hc.tq, hc.nres, 5 * 64, hc.nres)
    twin = hc.device(b, 1, first)                        # the same, in place
    ts = torch.from_numpy(sc).cuda()
    _, _, tk = b.evict_blocks(twin, ts, 5, 2, 64)
    assert torch.equal(keep, tk) and torch.equal(dst.first, twin.first)
    assert torch.equal(out[:, :hc.T], ts[:, :hc.T]) and not out[:, hc.T:].any()
    for x, y in zip((*dst.k[:3], *dst.v[:3]), (*twin.k[:3], *twin.v[:3])):
        assert torch.equal(x, y)
    # the padding that stays is not attended to
    q = torch.randn((3, 2, 4, 128), device="cuda").bfloat16()
    for a, c in zip(b.attend_chunk(q, dst), b.attend_chunk(q, twin)):
        assert torch.equal(a, c)


@pytest.mark.parametrize("shared", [(0,), (1, 2), (0, 1, 2)])
@pytest.mark.parametrize("which", ["k", "v"])
def test_caches_that_share_some_buffers(b, which, shared):
    """Buffers that dst shares with the source move in place, the others out of place."""
    import torch
    hc, sc, cache, ds = setup(b, 5)
    want = hc.device(b)
    ws = torch.from_numpy(sc).cuda()
    _, _, keep = b.evict_blocks(want, ws, 4, 1, 64)
    dst = hc.device(b)
    mine, theirs = list(getattr(dst, which)), getattr(cache, which)
    for m in shared:
        mine[m] = theirs[m]
    setattr(dst, which, tuple(mine))
    so = torch.zeros_like(ds)
    got = b.evict_blocks(cache, ds, 4, 1, 64, dst=dst, scores_out=so)
    assert torch.equal(got[2], keep) and torch.equal(so[:, :hc.T], ws[:, :hc.T])
    for x, y in zip((*dst.k[:3], *dst.v[:3]), (*want.k[:3], *want.v[:3])):
        assert torch.equal(x, y)


def test_a_store_without_channels(b):
    """C = 0: only the scores move, in more parts than a grid's second dimension holds."""
    import torch
    T, keep = 1 << 20, (1 << 20) - 3
    qp = b.QParams.sym(8, axis=b.ALONG_C, group=0, scale_dtype=b.F32)
    none = (torch.zeros(0, dtype=torch.uint8, device="cuda"),) + (None,) * 3
    cache = b.KVCache(k=none, v=none, shape=(1, T, 0), kqp=qp, vqp=qp, tq=T, nres=0, resid_rows=0)
    dst = b.KVCache(k=none, v=none, shape=(1, T, 0), kqp=qp, vqp=qp, tq=T, nres=0, resid_rows=0)
    sc = torch.arange(T, device="cuda", dtype=torch.float32)[None]
    _, out, ids = b.evict_blocks(cache, sc, keep, 0, 1, dst=dst, scores_out=torch.zeros_like(sc))
    assert torch.equal(ids[0].cpu(), torch.arange(3, T, dtype=torch.int32))
    assert torch.equal(out[0, :keep], sc[0, 3:]) and not out[0, keep:].any()


def test_an_empty_store_takes_any_block(b):
    """No block at all: the buffered tokens' scores stay, whatever the block's length."""
    import torch
    rng = np.random.default_rng(9)
    hc = S.HostCache(rng, 2, 128, 0, 128, 5, 64, *S.formats())
    for block in (64, 64 << 20, 64 << 34):
        cache = hc.device(b, 1, [0, 3])
        sc = torch.rand((2, 9), device="cuda")
        want = sc.clone()
        _, out, keep = b.evict_blocks(cache, sc, 4, 1, block)
        assert keep.shape == (2, 0) and (cache.tq, cache.nres) == (0, 5)
        assert torch.equal(out, want) and cache.first.tolist() == [0, 3]
