"""kvq_evict_blocks against its definition on the host: everything it writes is
moved or whole, so every comparison is exact."""
import numpy as np
import pytest

import oracle as O
import stream_util as S
from gpu_util import Guarded, kb

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def b():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return kb()


def expected(hc, sc, first, budget, window, block):
    """keep, scores, first and the six buffers after eviction, out of place onto copies."""
    nb = hc.tq // block
    kept, recent = min(budget, nb), min(window, nb)
    keep = np.zeros((hc.outer, kept), np.int32)
    out, f2 = sc.copy(), np.zeros(hc.outer, np.int32)
    bufs = [[None if a is None else a.copy() for a in c[:3]] for c in (hc.k, hc.v)]
    for o in range(hc.outer):
        s = [np.float64(sc[o, i * block:(i + 1) * block]).sum() for i in range(nb - recent)]
        rank = sorted(range(nb - recent), key=lambda i: (np.isnan(s[i]), -s[i] if not np.isnan(s[i]) else 0.0, i))
        ids = sorted(rank[:kept - recent] + list(range(nb - recent, nb)))
        keep[o] = ids
        tok = np.array([i * block + x for i in ids for x in range(block)], int)
        out[o, :kept * block] = sc[o, tok]
        out[o, kept * block:kept * block + hc.nres] = sc[o, hc.tq:hc.T]
        out[o, kept * block + hc.nres:hc.T] = 0
        f = max(first[o], 0) if first is not None else 0
        f2[o] = sum(min(max(f - i * block, 0), block) for i in ids) + max(f - hc.tq, 0)
        for (src, oq), dst in zip(((hc.k, hc.kq), (hc.v, hc.vq)), bufs):
            dst[0][o, :kept * block] = src[0][o, tok]
            per = block // oq.group if oq.axis == O.ALONG_T else block
            rows = np.array([i * per + x for i in ids for x in range(per)], int)
            for m in (1, 2):
                if src[m] is not None:
                    dst[m][o, :kept * per] = src[m][o, rows]
    return keep, out, f2, bufs


I8 = dict(scale_dtype=O.F32)
FORMATS = {
    "kivi": S.formats(),
    "two bits": S.formats(bits=2, kind="sym", gk=32, gv=32),
    "eight bits, per token, int8 zeros": tuple(
        O.QParams.asym(8, -128, 127, axis=O.ALONG_C, group=g, zero_dtype=O.I8, **I8) for g in (16, 0)),
    "float zeros": (O.QParams.asym(4, 0, 15, axis=O.ALONG_T, group=32, zero_dtype=O.F32, **I8),
                    O.QParams.sym(8, axis=O.ALONG_T, group=64)),
}
#   outer, C, tq, cap, nres, rows, block, budget, window, first
CASES = [
    ("kivi", (3, 128, 64 * 17, 64 * 17 + 40, 100, 192, 64, 16, 2, None)),
    ("kivi", (4, 128, 64 * 40, 64 * 41, 130, 192, 64, 9, 3, [0, 70, 2600, 5000])),
    ("kivi", (2, 128, 64 * 8, 64 * 8, 7, 64, 64, 8, 0, [3, 500])),        # nothing to evict
    ("kivi", (2, 128, 64 * 8, 64 * 8, 7, 64, 64, 100, 100, None)),        # more than there is
    ("kivi", (2, 64, 128 * 6, 128 * 6, 0, 0, 128, 1, 0, None)),           # two groups a block, one block stays
    ("kivi", (2, 64, 128 * 6, 128 * 6, 33, 40, 128, 2, 2, None)),         # the newest only
    ("kivi", (1, 128, 0, 128, 5, 64, 64, 4, 1, None)),                    # no block at all
    ("kivi", (1, 128, 64 * 1300, 64 * 1300, 5, 64, 64, 700, 10, None)),   # more blocks than threads
    ("kivi", (2, 64, 64 * 2300, 64 * 2304, 5, 64, 64, 1200, 10, [0, 7000])),   # more than are held in shared memory
    ("two bits", (3, 128, 32 * 21, 32 * 21 + 7, 50, 64, 32, 5, 1, None)),
    ("two bits", (2, 64, 96 * 5, 96 * 5, 3, 64, 96, 3, 1, [10, 200])),
    ("eight bits, per token, int8 zeros", (2, 48, 7 * 11, 80, 9, 16, 7, 4, 1, [9, 0])),
    ("eight bits, per token, int8 zeros", (1, 24, 40, 41, 3, 3, 1, 13, 5, None)),    # single tokens
    ("float zeros", (2, 40, 64 * 9, 64 * 9 + 1, 65, 70, 64, 4, 0, None)),
]


def scores_of(rng, kind, outer, n):
    if kind == "random":
        return np.exp(3 * rng.standard_normal((outer, n))).astype(np.float32)
    if kind == "ties":
        return rng.integers(0, 2, (outer, n)).astype(np.float32) * np.float32(0.5)
    if kind == "zeros":
        s = np.zeros((outer, n), np.float32)
        s[:, ::3] = -0.0
        return s
    s = rng.standard_normal((outer, n)).astype(np.float32) * 1e3             # signs, NaN, infinities
    s[rng.random((outer, n)) < 0.004] = np.nan
    s[rng.random((outer, n)) < 0.004] = np.inf
    s[rng.random((outer, n)) < 0.004] = -np.inf
    return s


@pytest.mark.parametrize("kind", ["random", "ties", "zeros", "odd"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_evict_blocks(b, case, kind):
    import torch
    fmt, (outer, C, tq, cap, nres, rows, block, budget, window, first) = CASES[case]
    rng = np.random.default_rng(case)
    hc = S.HostCache(rng, outer, C, tq, cap, nres, rows, *FORMATS[fmt])
    sc = scores_of(rng, kind, outer, hc.T + 3)
    keep, out, f2, bufs = expected(hc, sc, first, budget, window, block)

    for inplace in (False, True):
        cache = hc.device(b, 1, first)
        g = Guarded()
        if inplace:
            dst = cache
            ds = dso = torch.from_numpy(sc.copy()).cuda()
        else:
            dst = hc.device(b)                          # same garbage behind the blocks as the source has
            dst.k = tuple(None if t is None or m == 3 else _guarded(g, t) for m, t in enumerate(dst.k))
            dst.v = tuple(None if t is None or m == 3 else _guarded(g, t) for m, t in enumerate(dst.v))
            dst.first = torch.full((outer,), -7, dtype=torch.int32, device="cuda")
            ds = torch.from_numpy(sc).cuda()
            dso = _guarded(g, ds.view(torch.uint8).view(-1)).view(torch.float32).view(ds.shape)
        wB = b.kvq_evict_blocks_workspace(cache.shape, block)
        got = b.evict_blocks(cache, ds, budget, window, block, dst=dst, scores_out=dso, workspace=g.alloc(max(wB, 16)))
        g.check("kvq_evict_blocks")
        assert got[0] is dst and dst.tq == keep.shape[1] * block and dst.nres == nres
        assert np.array_equal(got[2].cpu().numpy(), keep)
        assert np.array_equal(dso.cpu().numpy().view(np.uint32), out.view(np.uint32))
        if first is not None or not inplace:
            assert np.array_equal(dst.first.cpu().numpy(), f2)
        for have, want in zip((dst.k, dst.v), bufs):
            for m in range(3):
                if want[m] is not None and want[m].size:
                    assert np.array_equal(have[m].cpu().numpy(), want[m].view(np.uint8).ravel()), (inplace, m)


def _guarded(g, t):
    w = g.alloc(max(t.numel(), 1))[:t.numel()] if t.numel() else t
    w.copy_(t)
    return w


def test_misaligned_buffers_move_too(b):
    """Stores at odd addresses (codes) and 2-byte addresses (metadata), in place."""
    import torch
    rng = np.random.default_rng(5)
    hc = S.HostCache(rng, 2, 128, 64 * 9, 64 * 9, 20, 64, *S.formats())
    sc = scores_of(rng, "random", 2, hc.T)
    keep, out, _, bufs = expected(hc, sc, None, 4, 1, 64)
    cache = hc.device(b)

    def shifted(t, by):
        big = torch.zeros(t.numel() + 16, dtype=torch.uint8, device="cuda")
        big[by:by + t.numel()] = t
        return big[by:by + t.numel()]
    cache.k = (shifted(cache.k[0], 3), shifted(cache.k[1], 2), shifted(cache.k[2], 6), cache.k[3])
    cache.v = (shifted(cache.v[0], 4), shifted(cache.v[1], 10), shifted(cache.v[2], 2), cache.v[3])
    _, got, kp = b.evict_blocks(cache, torch.from_numpy(sc).cuda(), 4, 1, 64)
    assert np.array_equal(kp.cpu().numpy(), keep) and np.array_equal(got.cpu().numpy(), out)
    for have, want in zip((cache.k, cache.v), bufs):
        for m in range(3):
            assert np.array_equal(have[m].cpu().numpy(), want[m].view(np.uint8).ravel()), m
