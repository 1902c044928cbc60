"""The forms of kvq_attend_chunk and kvq_attend_weights that only larger calls
take: query tiles that are split, whole tiles with a split tail, several jobs for
a CTA, several rounds of expansion; and formats that differ between K and V.

Everything is compared with the formulas in binary64 over the rows of
kvq_dequantize, with the tolerances of test_stream_attend_gpu.py (u = 2^-8, the
largest relative error of a rounding to bf16; e twice the logits' error):
  lse: e + (T + 64) 2^-23 + 4 2^-23 (|lse| + 1)
  out: (u + e + (T + 64) 2^-23) sum_t p_t |v_t| + u |out|
  weights: (e + (rows + 64) 2^-23 + 8 2^-23 |lse|) sum w + 2^-23 |score|
"""
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


# ---- the plans, restated, so that a case is known to take the form it is here for

def query_tiles(outer, T, rows):
    """(tiles of 256 rows taken whole, split tiles, splits of each)"""
    tiles, keys = outer * -(-rows // 256), -(-T // 128)
    plan, best = (tiles, 0, 1), -(-tiles // 152) * (keys + 6)
    s = 2
    while s * 2 <= keys and tiles * s <= 608:
        cost = -(-tiles * s // 152) * (-(-keys // s) + 6) + 8
        if cost < best:
            plan, best = (0, tiles, s), cost
        s += 1
    tail = tiles % 152
    s = min(152 // tail, keys // 2) if tail else 1
    if tiles > 152 and s > 1 and tiles // 152 * (keys + 6) + -(-keys // s) + 14 < best:
        plan = (tiles - tail, tail, s)
    return plan


def weight_jobs(outer, T, rows):
    """(jobs, splits of the rows)"""
    jobs, tiles = outer * -(-T // 256), -(-rows // 128)
    best, plan, s = None, 1, 1
    while s == 1 or (s <= tiles and jobs * s <= 8 * 152):
        cost = -(-jobs * s // 152) * max(-(-tiles // s) + 1, 3)
        if best is None or cost < best:
            best, plan = cost, s
        s += 1
    return jobs * plan, plan


def make(b, seed, B, H, G, n, C, T, R=60, bits=4, first=None, loud=1.0):
    """(cache, q, K, V): rows in binary64 on the GPU; hidden rows are zero there and NaN in the cache's buffers."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    qp = [b.QParams.asym(bits, 0, (1 << bits) - 1, axis=a, group=64, residual=R, scale_dtype=b.BF16, zero_dtype=b.BF16)
          for a in (b.ALONG_T, b.ALONG_C)]
    kv = [b.quantize(torch.randn((B * H, T, C), generator=gen, device="cuda").bfloat16(), p) for p in qp]
    rows = [b.dequantize(t).double() for t in kv]
    f = None
    if first is not None:
        first = [first[o % len(first)] for o in range(B * H)]
        f = torch.tensor(first, dtype=torch.int32, device="cuda")
        scale = kv[1].scale.view(torch.bfloat16).view(B * H, T - R, C // 64)
        for o, x in enumerate(first):
            for r in rows:
                r[o, :x] = 0
            scale[o, :min(x, T - R)] = float("nan")
    q = (loud * torch.randn((B, n, H * G, C), generator=gen, device="cuda")).bfloat16()
    return b.KVCache.from_quantized(*kv, kv_heads=H, first=f), q, *rows


def slice_rows(t, o, H):
    """[n, group, ...] of slice o from [B, n, H * group, ...]"""
    G = t.shape[2] // H
    return t[o // H, :, (o % H) * G:(o % H + 1) * G]


def solve(cache, q, K, V, o):
    """p, lse, e, out, sum p|v| of slice o, rows [n, group]"""
    import torch
    n, C, T = q.shape[1], q.shape[3], cache.T
    qs = slice_rows(q, o, cache.kv_heads).double()
    x = torch.einsum("ijc,tc->ijt", qs, K[o]) / C ** 0.5
    mag = torch.einsum("ijc,tc->ijt", qs.abs(), K[o].abs()) / C ** 0.5
    t = torch.arange(T, device=q.device)
    seen = (t <= T - n + torch.arange(n, device=q.device)[:, None])[:, None]
    if cache.first is not None:
        seen = seen & (t >= cache.first[o])
    x, mag = torch.where(seen, x, -float("inf")), torch.where(seen, mag, 0.0)
    lse = torch.logsumexp(x, -1)
    p = torch.where(seen, torch.exp(x - torch.where(lse.isinf(), 0.0, lse)[..., None]), 0.0)
    big = torch.where(x.isinf(), 0.0, x.abs()).amax(-1)
    e = 2 * ((C + 8) * 2.0 ** -23 * mag.amax(-1) + 8 * 2.0 ** -23 * (big + 1.0))       # stream_util.logit_error
    return p, lse, e, torch.einsum("ijt,tc->ijc", p, V[o]), torch.einsum("ijt,tc->ijc", p, V[o].abs())


def check_attend(cache, q, K, V, out, lse, slices=None):
    T, u = cache.T, 2.0 ** -8
    for o in slices if slices is not None else range(cache.shape[0]):
        p, wl, e, want, absout = solve(cache, q, K, V, o)
        got, gl = slice_rows(out, o, cache.kv_heads).double(), slice_rows(lse, o, cache.kv_heads).double()
        none = wl.isinf()
        assert bool((gl.isneginf() == none).all()) and bool((got[none] == 0).all())
        tl = e + (T + 64) * 2.0 ** -23 + 4 * 2.0 ** -23 * (wl.abs() + 1)
        assert bool(((gl - wl).abs() <= tl)[~none].all()), o
        to = (u + e + (T + 64) * 2.0 ** -23)[..., None] * absout + u * want.abs() + 1e-30
        assert bool(((got - want).abs() <= to).all()), o


def check_weights(cache, q, K, V, lse, scores, got, slices=None):
    """lse: the float32 values that the call was given"""
    import torch
    T, rows = cache.T, q.shape[1] * q.shape[2] // cache.kv_heads
    for o in slices if slices is not None else range(cache.shape[0]):
        p, wl, e, _, _ = solve(cache, q, K, V, o)
        l32 = slice_rows(lse, o, cache.kv_heads).double()
        none = wl.isinf()
        w = p * torch.exp(torch.where(none, 0.0, wl - l32))[..., None]       # exp(x - lse) of the lse given
        tol = torch.einsum("ijt,ij->t", w, e + (rows + 64) * 2.0 ** -23 + 8 * 2.0 ** -23 * torch.where(none, 0.0, wl.abs()))
        want = scores[o, :T].double() + w.sum((0, 1))
        assert bool(((got[o, :T].double() - want).abs() <= tol + 2.0 ** -23 * want.abs() + 1e-30).all()), o


#   batch, kv_heads, group, n, C, T, more, whole tiles?, split tiles?
ATTEND = {
    "up to 256 rows, split": ((1, 2, 4, 20, 128, 4196), dict(first=[0, 1500]), False, True),
    "up to 256 rows, split, two bits, C 64": ((1, 1, 8, 25, 64, 4196), dict(bits=2), False, True),
    "up to 256 rows, whole and split tiles": ((12, 13, 4, 50, 128, 2100), dict(first=[0, 3, 700]), True, True),
    "up to 256 rows, two bits, whole and split tiles": ((4, 40, 4, 40, 64, 3000), dict(bits=2), True, True),
    "many rows, whole and split tiles": ((2, 10, 4, 512, 128, 2148), {}, True, True),
    "many rows, C 64, whole and split tiles": ((3, 11, 5, 220, 64, 2148), dict(first=[0, 200, 1999, 2148]), True, True),
}
#   batch, kv_heads, group, n, C, T, more, splits of the rows?
WEIGHTS = {
    "many jobs": ((2, 8, 4, 20, 128, 5200), dict(first=[0, 300, 2600, 5200, 4990]), False),
    "many jobs, two row tiles": ((4, 5, 6, 40, 64, 5200), dict(bits=2), False),
    "many jobs, split rows": ((2, 8, 4, 250, 128, 5200), dict(first=[0, 0, 2700]), True),
    "many jobs, many rows": ((2, 9, 2, 1500, 64, 4700), dict(first=[0, 4600, 0, 4700, 0, 0, 1024]), None),
}


@pytest.mark.parametrize("name", ATTEND)
def test_attend_over_query_tile_plans(b, name):
    import torch
    (B, H, G, n, C, T), more, whole, split = ATTEND[name]
    plan = query_tiles(B * H, T, n * G)
    assert (plan[0] > 0, plan[1] > 0 and plan[2] > 1) == (whole, split), plan
    cache, q, K, V = make(b, len(name), B, H, G, n, C, T, **more)
    out, lse = b.attend_chunk(q, cache)
    check_attend(cache, q, K, V, out, lse)
    again = b.attend_chunk(q, cache)
    assert torch.equal(again[0].view(torch.int16), out.view(torch.int16)) and torch.equal(again[1], lse)


@pytest.mark.parametrize("name", WEIGHTS)
def test_weights_over_many_jobs(b, name):
    import torch
    (B, H, G, n, C, T), more, split = WEIGHTS[name]
    jobs, splits = weight_jobs(B * H, T, n * G)
    assert jobs > 2 * 152 and (split is None or split == (splits > 1)), (jobs, splits)
    cache, q, K, V = make(b, len(name), B, H, G, n, C, T, **more)
    _, lse = b.attend_chunk(q, cache)
    gen = torch.Generator(device="cuda").manual_seed(1)
    scores = torch.rand((B * H, T + 3), generator=gen, device="cuda")
    got = b.attend_weights(q, lse, cache, scores, torch.full_like(scores, -1.0))
    assert bool((got[:, T:] == -1.0).all())
    check_weights(cache, q, K, V, lse, scores, got)
    assert torch.equal(b.attend_weights(q, lse, cache, scores)[:, :T], got[:, :T])


# a case for each plan of both calls
BOTH = [ATTEND["up to 256 rows, split"], ATTEND["up to 256 rows, whole and split tiles"],
        ATTEND["many rows, whole and split tiles"], WEIGHTS["many jobs, split rows"]]


@pytest.mark.parametrize("case", range(len(BOTH)))
def test_plans_under_capture(b, case):
    """Both calls in one graph with workspaces of their own; replays see new queries."""
    import torch
    (B, H, G, n, C, T), more = BOTH[case][:2]
    cache, q, _, _ = make(b, case, B, H, G, n, C, T, **more)
    wa, ww = (torch.empty(max(f(cache.shape, cache.resid_rows, n, G), 1), dtype=torch.uint8, device="cuda")
              for f in (b.kvq_attend_chunk_workspace, b.kvq_attend_weights_workspace))
    out, lse = b.attend_chunk(q, cache, workspace=wa)
    sc = torch.zeros((B * H, T), device="cuda")
    b.attend_weights(q, lse, cache, sc, sc, ww)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.attend_chunk(q, cache, out, lse, wa)
        b.attend_weights(q, lse, cache, sc, sc, ww)
    q.copy_(torch.randn_like(q.float()).bfloat16())
    sc.zero_()
    graph.replay()
    graph.replay()
    want, wl = b.attend_chunk(q, cache)
    one = b.attend_weights(q, wl, cache)
    torch.cuda.synchronize()
    assert torch.equal(out.view(torch.int16), want.view(torch.int16)) and torch.equal(lse, wl)
    assert torch.equal(sc, one + one)


@pytest.mark.parametrize("case", range(len(BOTH)))
def test_plans_on_two_streams(b, case):
    import torch
    (B, H, G, n, C, T), more = BOTH[case][:2]
    cache, q, _, _ = make(b, case, B, H, G, n, C, T, **more)
    want, wl = b.attend_chunk(q, cache)
    ww = b.attend_weights(q, wl, cache)
    torch.cuda.synchronize()
    st = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [(b.attend_chunk(q, cache, stream=s), b.attend_weights(q, wl, cache, stream=s)) for _ in range(3) for s in st]
    torch.cuda.synchronize()
    for (o, l), w in got:
        assert torch.equal(o.view(torch.int16), want.view(torch.int16)) and torch.equal(l, wl) and torch.equal(w, ww)


def test_rounds_of_expansion(b):
    """Over 1 GiB of expanded rows, so several rounds of slices.  Queries loud enough that a few tokens carry the
    weight, and values with an offset of their own for every slice and channel: outputs are of order one, and another
    slice's values, or another tile's, do not pass."""
    import torch
    outer, T, C, n, G = 20, 112000, 128, 80, 4
    per_round = (1 << 30) // (-(-T // 128) * 128 * C * 4)
    assert 1 < per_round < outer
    gen = torch.Generator(device="cuda").manual_seed(7)
    kq, vq = (b.QParams.asym(4, 0, 15, axis=a, group=64, scale_dtype=b.BF16, zero_dtype=b.BF16) for a in (b.ALONG_T, b.ALONG_C))
    at = torch.arange(outer, device="cuda")[:, None] * 5 + torch.arange(C, device="cuda") * 3
    offset = ((at % 17).float() - 8) / 4
    k, v = (b.quantize((torch.randn((outer, T, C), generator=gen, device="cuda") + add).bfloat16(), qp)
            for qp, add in ((kq, 0.0), (vq, offset[:, None])))
    cache = b.KVCache.from_quantized(k, v, kv_heads=outer // 2)
    q = (4 * torch.randn((2, n, outer // 2 * G, C), generator=gen, device="cuda")).bfloat16()
    out, lse = b.attend_chunk(q, cache)
    K, V = b.dequantize(k), b.dequantize(v)

    class Rows:                                          # binary64 of one slice at a time
        def __init__(self, t):
            self.t = t

        def __getitem__(self, o):
            return self.t[o].double()
    check = [0, 9, per_round - 1, per_round, outer - 1]
    some = slice(n - 6, n)                                # the last queries' rows: the others are read alike
    cut, lcut = out[:, some].contiguous(), lse[:, some].contiguous()
    qcut = q[:, some].contiguous()
    check_attend(cache, qcut, Rows(K), Rows(V), cut, lcut, check)
    with pytest.raises(AssertionError):                  # another slice's values
        check_attend(cache, qcut, Rows(K), Rows(V.roll(1, 0)), cut, lcut, check[:1])
    with pytest.raises(AssertionError):                  # another tile's values
        check_attend(cache, qcut, Rows(K), Rows(V.roll(128, 1)), cut, lcut, check[:1])
    assert bool(out.isfinite().all()) and bool((out.float().abs().amax(-1) > 0.1).all())


KINDS = ["asym", "sym", "signed"]


@pytest.mark.parametrize("bits", [2, 4])
@pytest.mark.parametrize("n", [1, 4, 20, 150])
@pytest.mark.parametrize("kinds", [(k, v) for k in KINDS for v in KINDS if k != v])
def test_keys_and_values_of_different_kinds(b, kinds, n, bits):
    """symmetric keys with asymmetric values, signed with unsigned codes, and the reverse"""
    import torch
    B, H, G, C, tq, nres = 1, 2, 4, 128, 384, 40
    rng = np.random.default_rng(n + 10 * bits)
    kq, vq = S.formats(bits=bits, kind=kinds[0])[0], S.formats(bits=bits, kind=kinds[1], gv=32)[1]
    hc = S.HostCache(rng, B * H, C, tq, tq + 64, nres, 64, kq, vq)
    bits16 = S.W.to_bf16_bits(rng.standard_normal((B, n, H * G, C)).astype(np.float32))
    q = torch.from_numpy(bits16.view(np.int16).copy()).view(torch.bfloat16).cuda()
    cache = hc.device(b, H)
    K, V = (torch.from_numpy(r).cuda() for r in (hc.K, hc.V))
    out, lse = b.attend_chunk(q, cache)
    check_attend(cache, q, K, V, out, lse)
    zero = torch.zeros((B * H, hc.T), device="cuda")
    check_weights(cache, q, K, V, lse, zero, b.attend_weights(q, lse, cache))


# a case for each form: one split, a cluster, the workspace, fused, expanded, whole tiles and a split tail
IN_PLACE = [(2, 70, 4, 1, 128, 100), (1, 2, 4, 2, 128, 1000), (1, 2, 8, 4, 64, 9000), (1, 2, 4, 20, 128, 500),
            (1, 2, 4, 130, 128, 400), *(c[0] for c in BOTH[:3])]


@pytest.mark.parametrize("case", range(len(IN_PLACE)))
def test_out_in_place_of_the_queries(b, case):
    import torch
    cache, q, _, _ = make(b, case, *IN_PLACE[case])
    want, wl = b.attend_chunk(q, cache)
    got, lse = b.attend_chunk(q, cache, out=q)
    assert got is q and torch.equal(q.view(torch.int16), want.view(torch.int16)) and torch.equal(lse, wl)


def test_offsets_past_32_bits(b):
    """A store of 5.4 billion values each of K and V: every form of the three calls, the first and the last slice
    checked."""
    import torch
    outer, H, T, C, block = 40, 8, 1 << 20, 128, 64
    assert outer * T * C > 1 << 32 and outer * T * C // 2 > 1 << 31
    gen = torch.Generator(device="cuda").manual_seed(3)
    kv, rows = [], []
    for axis in (b.ALONG_T, b.ALONG_C):
        qp = b.QParams.asym(4, 0, 15, axis=axis, group=block, scale_dtype=b.BF16, zero_dtype=b.BF16)
        t = b.quantize(torch.randn((outer, T, C), generator=gen, device="cuda", dtype=torch.bfloat16), qp)
        x = b.dequantize(t)
        rows.append({o: x[o].double() for o in (0, outer - 1)})
        kv.append(t)
        del x
    cache = b.KVCache.from_quantized(*kv, kv_heads=H)
    for n, G in ((1, 4), (3, 4), (4, 8), (20, 4), (75, 4)):
        q = (3 * torch.randn((outer // H, n, H * G, C), generator=gen, device="cuda")).bfloat16()
        out, lse = b.attend_chunk(q, cache)
        check_attend(cache, q, *rows, out, lse, (0, outer - 1))
        got = b.attend_weights(q, lse, cache)
        zero = torch.zeros((outer, T), device="cuda")
        check_weights(cache, q, *rows, lse, zero, got, (0, outer - 1))
    old = [t.codes.view(outer, T, C // 2)[-1].clone() for t in kv]
    scores = torch.rand((outer, T), generator=gen, device="cuda")
    sums = scores[-1].view(-1, block).double().sum(1)
    keep = b.evict_blocks(cache, scores, 1000, 0, block)[2][-1].long()
    assert torch.equal(keep, torch.sort(torch.topk(sums, 1000).indices).values)
    tok = (keep[:, None] * block + torch.arange(block, device="cuda")).flatten()
    for t, was in zip(kv, old):
        assert torch.equal(t.codes.view(outer, T, C // 2)[-1, :len(tok)], was[tok])
