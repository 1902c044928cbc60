"""kvq_attend_chunk and kvq_attend_weights against the formulas in binary64.

Both sides read the same quantized cache, whose rows are exactly those of
kvq_dequantize, so only the attention's own arithmetic differs.  Tolerances
(u = 2^-8, the largest relative error of a rounding to bf16; logit errors from
stream_util.logit_error, e = twice that of the row: a probability is the
exponential of a difference of two):
  lse:     e + (T + 64) 2^-23 + 4 2^-23 (|lse| + 1)
           (float32 sums of positive terms, at most one rounding a token and a
           few a merge; the logarithm and its scaling);
  out:     (u + e + (T + 64) 2^-23) sum_t p_t |v_t| + u |out|
           (p rounded to bf16 for the value product, float32 sums, out rounded);
  weights: (e + (rows + 64) 2^-23 + 8 2^-23 |lse|) sum w + 2^-23 |score|.
"""
import zlib

import numpy as np
import pytest

import stream_util as S
from gpu_util import Guarded, kb

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def b():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return kb()


#   batch, kv_heads, group, n, C, tq, cap, nres, rows, formats, extras
CASES = {
    "one token alone": (1, 1, 1, 1, 128, 0, 64, 1, 64, {}, {}),
    "buffer only": (2, 2, 4, 1, 128, 0, 0, 37, 64, {}, {}),
    "store only, one block": (1, 2, 8, 1, 128, 64, 64, 0, 0, {}, {}),
    "empty cache": (2, 1, 4, 3, 128, 0, 64, 0, 64, {}, {}),
    "more queries than tokens": (1, 2, 3, 9, 64, 0, 64, 5, 64, {}, {}),
    "ordinary step": (2, 2, 8, 1, 128, 960, 1024, 77, 192, {}, {}),
    "step of 16 heads": (1, 2, 16, 1, 128, 512, 640, 130, 192, {}, {}),
    "step of 64 heads": (1, 1, 64, 1, 64, 192, 192, 31, 64, {}, {}),
    "ragged store end": (1, 2, 4, 2, 128, 333, 333, 19, 19, dict(gk=96), {}),
    "two bits, symmetric": (1, 2, 4, 5, 128, 640, 704, 66, 192, dict(bits=2, kind="sym", gk=32, gv=128), {}),
    "two bits, C 64": (1, 3, 5, 2, 64, 448, 448, 10, 64, dict(bits=2, gv=32), {}),
    "symmetric, C 64": (2, 1, 7, 3, 64, 256, 320, 33, 64, dict(kind="sym", gk=128), {}),
    "signed zero points": (1, 2, 4, 4, 128, 320, 320, 63, 64, dict(kind="signed", gk=32, gv=32), {}),
    "far zero points": (1, 2, 4, 3, 128, 256, 256, 20, 64, {}, dict(shift=100.0)),
    "far zero points, two bits": (1, 1, 2, 1, 64, 256, 256, 0, 64, dict(bits=2), dict(shift=-30.0)),
    "far zero points, symmetric": (1, 1, 2, 2, 64, 128, 256, 40, 64, dict(kind="sym"), dict(shift=50.0)),
    "padding": (4, 2, 4, 40, 128, 256, 320, 50, 64, {}, dict(first=[0, 0, -5, 1, 100, 290, 306, 999])),
    "padding, step": (5, 1, 8, 1, 128, 256, 320, 50, 64, {}, dict(first=[0, 31, 32, 305, 400])),
    "padding, extreme": (3, 1, 4, 2, 128, 256, 256, 50, 64, {}, dict(first=[2**31 - 1, -2**31, 306])),
    "padding, extreme, many rows": (3, 1, 8, 40, 64, 256, 256, 50, 64, dict(gv=32), dict(first=[2**31 - 1, -2**31, 305])),
    "padding, extreme, prompt": (3, 1, 8, 50, 128, 256, 256, 50, 64, {}, dict(first=[2**31 - 1, -2**31, 200])),
    "prompt from nothing": (1, 2, 2, 300, 64, 256, 256, 44, 64, {}, {}),
    "prompt, odd group": (1, 1, 3, 517, 128, 448, 448, 69, 128, {}, {}),
    "chunk": (1, 2, 4, 130, 128, 2048, 2112, 100, 192, {}, {}),
    "chunk, padded": (2, 1, 5, 70, 128, 1024, 1024, 101, 192, {}, dict(first=[3, 700])),
    "long, split": (1, 2, 4, 1, 128, 9024, 9088, 100, 192, {}, {}),
    "long, split, padded": (1, 2, 1, 2, 64, 9024, 9088, 100, 192, {}, dict(first=[8000, 9100])),
    "many rows, two bits": (1, 2, 4, 40, 128, 640, 704, 66, 192, dict(bits=2, gk=32, gv=128), {}),
    "many rows, two bits, C 64": (1, 2, 8, 20, 64, 448, 448, 10, 64, dict(bits=2, kind="sym", gv=32), {}),
    "many rows, far zero points": (1, 1, 5, 30, 128, 512, 512, 40, 64, {}, dict(shift=100.0)),
    "many rows, symmetric, C 64": (2, 1, 2, 50, 64, 512, 576, 33, 64, dict(kind="sym", gk=128), {}),
    "many rows, ragged store": (1, 2, 7, 33, 128, 333, 333, 19, 19, dict(gk=96, gv=32), {}),
    "many rows, signed, padded": (3, 1, 16, 9, 128, 480, 512, 64, 64, dict(kind="signed", gk=32), dict(first=[0, 200, 543])),
    "many rows, split": (1, 1, 8, 40, 128, 4096, 4096, 100, 192, {}, dict(first=[1500])),
    "more rows than tokens": (1, 2, 4, 70, 128, 0, 64, 50, 64, {}, {}),
    "prompt, two bits": (1, 1, 4, 200, 128, 512, 576, 30, 64, dict(bits=2, gk=32, gv=32), {}),
    "prompt, two bits, C 64": (1, 1, 4, 200, 64, 512, 576, 30, 64, dict(bits=2, kind="sym"), {}),
    "prompt, far zero points": (1, 1, 3, 250, 128, 320, 320, 30, 64, {}, dict(shift=-60.0)),
    "prompt, padded": (3, 1, 4, 150, 128, 333, 333, 60, 64, dict(gk=96), dict(first=[0, 130, 390])),
    "many rows, empty cache": (2, 1, 4, 20, 128, 0, 64, 0, 64, {}, {}),
    "prompt, empty cache": (1, 1, 4, 100, 64, 0, 64, 0, 64, {}, {}),
    "rows of 24": (1, 2, 8, 3, 128, 512, 512, 40, 64, {}, {}),
    "rows of 32, two bits": (2, 1, 16, 2, 64, 384, 384, 40, 64, dict(bits=2), dict(first=[0, 77])),
    "rows of 33": (1, 1, 33, 1, 128, 256, 256, 40, 64, {}, {}),
    "rows of 256": (1, 1, 64, 4, 128, 640, 640, 40, 64, {}, {}),
    "rows of 257": (1, 1, 1, 257, 128, 640, 640, 40, 64, {}, {}),
    "loud": (1, 1, 4, 6, 128, 512, 512, 64, 64, {}, dict(scale=6.0)),
}


def build(name):
    rng = np.random.default_rng(zlib.crc32(name.encode()))
    B, H, G, n, C, tq, cap, nres, rows, fm, ex = CASES[name]
    kq, vq = S.formats(**{"gv": 64, **fm})
    hc = S.HostCache(rng, B * H, C, tq, cap, nres, rows, kq, vq, ex.get("shift", 0.0), ex.get("scale", 1.0))
    first = ex.get("first")
    if first is not None:
        # what lies wholly in the padding may be anything: NaN scales, NaN rows
        for o, f in enumerate(first):
            f = min(max(f, 0), hc.T)
            hc.k[1][o, :min(f, tq) // kq.group] = 0x7FC0
            hc.v[1][o, :min(f, tq)] = 0x7FC0
            if f > tq:
                hc.k[3][o, :f - tq] = hc.v[3][o, :f - tq] = 0x7FC0
    q = S.W.to_bf16_bits(rng.standard_normal((B, n, H * G, C)).astype(np.float32))
    return hc, q, first


def upload_bf16(bits):
    import torch
    return torch.from_numpy(bits.view(np.int16).copy()).view(torch.bfloat16).cuda()


def visible(hc, first):
    """K and V with every hidden row zeroed (binary64 NaN would spread)."""
    K, V = hc.K.copy(), hc.V.copy()
    for o, f in enumerate(first if first is not None else []):
        K[o, :max(f, 0)] = 0.0
        V[o, :max(f, 0)] = 0.0
    return K, V


def reference(hc, q, first, kv_heads):
    K, V = visible(hc, first)
    x, mag = S.logits(S.bf16_to_f64(q), K, first, kv_heads)
    p, lse = S.softmax(x)
    out = np.einsum("oijt,otc->oijc", p, V)
    absout = np.einsum("oijt,otc->oijc", p, np.abs(V))
    return x, mag, p, lse, out, absout


@pytest.mark.parametrize("name", CASES)
def test_attend_chunk(b, name):
    import torch
    hc, q, first = build(name)
    B, H, G, n, C = CASES[name][:5]
    x, mag, p, lse, out, absout = reference(hc, q, first, H)
    cache = hc.device(b, H, first)
    g = Guarded()
    do = g.alloc(max(q.size * 2, 16)).view(torch.bfloat16)[:q.size].view(q.shape)
    dl = g.alloc(max(q.size // C * 4, 16)).view(torch.float32)[:q.size // C].view(q.shape[:3])
    wB = b.kvq_attend_chunk_workspace(cache.shape, cache.resid_rows, n, G)
    b.attend_chunk(upload_bf16(q), cache, do, dl, g.alloc(max(wB, 16)))
    g.check("kvq_attend_chunk")
    got, gl = do.float().cpu().numpy().astype(np.float64), dl.cpu().numpy().astype(np.float64)
    e = 2 * S.logit_error(mag, x, C)
    want, wl = S.to_rows(out, H), S.to_rows(lse, H)
    none = np.isinf(wl)
    assert np.array_equal(np.isneginf(gl), none)
    assert np.all(got[none] == 0.0)
    tl = S.to_rows(e, H) + (hc.T + 64) * 2.0 ** -23 + 4 * 2.0 ** -23 * (np.abs(wl) + 1)
    assert np.all(np.abs(gl[~none] - wl[~none]) <= tl[~none]), np.max(np.abs(gl[~none] - wl[~none]) / tl[~none])
    u = 2.0 ** -8
    to = S.to_rows((u + e[..., None] + (hc.T + 64) * 2.0 ** -23) * absout, H) + u * np.abs(want) + 1e-30
    assert np.all(np.isfinite(got))
    assert np.all(np.abs(got - want) <= to), np.max(np.abs(got - want) / to)
    again = b.attend_chunk(upload_bf16(q), cache)           # equal calls give equal bits, lse optional
    assert torch.equal(again[0].view(torch.int16), do.view(torch.int16)) and torch.equal(again[1], dl)


@pytest.mark.parametrize("name", CASES)
def test_attend_weights(b, name):
    import torch
    hc, q, first = build(name)
    B, H, G, n, C = CASES[name][:5]
    x, mag, p, lse, _, _ = reference(hc, q, first, H)
    rng = np.random.default_rng(1)
    stride = hc.T + 5
    sc = rng.random((B * H, stride)).astype(np.float32)
    l32 = lse.astype(np.float32)
    with np.errstate(invalid="ignore"):
        w = np.where(np.isinf(x), 0.0, np.exp(x - l32[..., None].astype(np.float64)))
    w = np.where(np.isinf(l32)[..., None], 0.0, w)
    e = 2 * S.logit_error(mag, x, C) + (n * G + 64) * 2.0 ** -23 + 8 * 2.0 ** -23 * np.where(np.isinf(lse), 0, np.abs(lse))
    tol = np.einsum("oijt,oij->ot", w, e) + 2.0 ** -23 * (sc[:, :hc.T] + w.sum((1, 2))) + 1e-30
    cache = hc.device(b, H, first)
    dq, dl = upload_bf16(q), torch.from_numpy(S.to_rows(l32, H).copy()).cuda()
    g = Guarded()
    out = g.alloc(max(sc.size * 4, 16)).view(torch.float32)[:sc.size].view(sc.shape)
    before = out.clone()
    wB = b.kvq_attend_weights_workspace(cache.shape, cache.resid_rows, n, G)
    ds = torch.from_numpy(sc).cuda()
    b.attend_weights(dq, dl, cache, ds, out, g.alloc(max(wB, 16)))
    g.check("kvq_attend_weights")
    got = out.cpu().numpy()[:, :hc.T].astype(np.float64)
    assert torch.equal(out[:, hc.T:].view(torch.int32), before[:, hc.T:].view(torch.int32))
    want = sc[:, :hc.T].astype(np.float64) + w.sum((1, 2))
    assert np.all(np.abs(got - want) <= tol), np.max(np.abs(got - want) / tol)
    inplace = ds.clone()
    b.attend_weights(dq, dl, cache, inplace, inplace)
    assert torch.equal(inplace[:, :hc.T], out[:, :hc.T]) and torch.equal(inplace[:, hc.T:], ds[:, hc.T:])
    bare = b.attend_weights(dq, dl, cache).cpu().numpy().astype(np.float64)
    assert np.all(np.abs(bare - w.sum((1, 2))) <= tol)


# one case for each form: few rows in a cluster and through the workspace, up to 256 rows, more
FORMS = ["ordinary step", "long, split", "many rows, split", "chunk"]


@pytest.mark.parametrize("name", FORMS)
def test_a_captured_call_replays_on_new_data(b, name):
    """attend_chunk and attend_weights in one graph: replay sees new queries."""
    import torch
    hc, q, first = build(name)
    B, H, G, n = CASES[name][:4]
    cache = hc.device(b, H, first)
    dq = upload_bf16(q)
    out, lse = b.attend_chunk(dq, cache)
    wa, ww = (torch.empty(max(f(cache.shape, cache.resid_rows, n, G), 1), dtype=torch.uint8, device="cuda")
              for f in (b.kvq_attend_chunk_workspace, b.kvq_attend_weights_workspace))
    sc = torch.zeros((B * H, hc.T), device="cuda")
    b.attend_weights(dq, lse, cache, sc, sc, ww)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.attend_chunk(dq, cache, out, lse, wa)
        b.attend_weights(dq, lse, cache, sc, sc, ww)
    dq.copy_(torch.randn_like(dq.float()).bfloat16())
    sc.zero_()
    graph.replay()
    graph.replay()
    want, wl = b.attend_chunk(dq, cache)
    one = b.attend_weights(dq, wl, cache)
    torch.cuda.synchronize()
    assert torch.equal(out.view(torch.int16), want.view(torch.int16)) and torch.equal(lse, wl)
    assert torch.equal(sc, one + one)


@pytest.mark.parametrize("name", FORMS)
def test_other_streams(b, name):
    """Calls that may overlap on two streams, each with its own workspace and outputs."""
    import torch
    hc, q, first = build(name)
    cache = hc.device(b, CASES[name][1], first)
    dq = upload_bf16(q)
    want, wl = b.attend_chunk(dq, cache)
    ww = b.attend_weights(dq, wl, cache)
    torch.cuda.synchronize()
    st = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [(b.attend_chunk(dq, cache, stream=s), b.attend_weights(dq, wl, cache, stream=s)) for _ in range(4) for s in st]
    torch.cuda.synchronize()
    for (o, l), w in got:
        assert torch.equal(o.view(torch.int16), want.view(torch.int16)) and torch.equal(l, wl) and torch.equal(w, ww)


def test_from_quantized_agrees_with_dequantize(b):
    """A cache of two quantize() calls: the plain attention over dequantize()'s rows."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(3)
    k, v = (torch.randn((4, 700, 128), generator=gen, device="cuda").bfloat16() for _ in range(2))
    kq = b.QParams.asym(4, 0, 15, axis=b.ALONG_T, group=64, residual=60, scale_dtype=b.BF16, zero_dtype=b.BF16)
    vq = b.QParams.asym(4, 0, 15, axis=b.ALONG_C, group=64, residual=60, scale_dtype=b.BF16, zero_dtype=b.BF16)
    qk, qv = b.quantize(k, kq), b.quantize(v, vq)
    q = torch.randn((2, 1, 8, 128), generator=gen, device="cuda").bfloat16()
    out, lse = b.attend_chunk(q, b.KVCache.from_quantized(qk, qv, kv_heads=2))
    K, V = b.dequantize(qk).double(), b.dequantize(qv).double()
    x = torch.einsum("ojc,otc->ojt", q.reshape(4, 4, 128).double(), K) / 128 ** 0.5
    p = torch.softmax(x, -1)
    want = p @ V
    tol = 2.0 ** -8 * (want.abs() + p @ V.abs()) + 1e-4
    assert bool(((out.reshape(4, 4, 128).double() - want).abs() <= tol).all())
    assert bool(((lse.reshape(4, 4).double() - torch.logsumexp(x, -1)).abs() <= 1e-4).all())


def test_more_slices_than_are_expanded_at_once(b):
    """Over 1 GiB of expanded rows: several rounds of slices.  The last queries of
    the chunk are also asked for alone, which takes the kernel of few rows."""
    import torch
    outer, T, C, n, G = 20, 112000, 128, 80, 4
    assert outer * T * C * 4 > 1 << 30
    gen = torch.Generator(device="cuda").manual_seed(7)
    kq, vq = (b.QParams.asym(4, 0, 15, axis=a, group=64, scale_dtype=b.BF16, zero_dtype=b.BF16) for a in (b.ALONG_T, b.ALONG_C))
    k, v = (b.quantize(torch.randn((outer, T, C), generator=gen, device="cuda").bfloat16(), qp) for qp in (kq, vq))
    cache = b.KVCache.from_quantized(k, v, kv_heads=outer // 2)
    q = torch.randn((2, n, outer // 2 * G, C), generator=gen, device="cuda").bfloat16()
    out, lse = b.attend_chunk(q, cache)
    few, fl = b.attend_chunk(q[:, -8:].contiguous(), cache)
    # both are within u (sum p |v| + |out|) of the same value, u = 2^-8, and |v| <= 6 here
    assert bool(((out[:, -8:].float() - few.float()).abs() <= 2 * 2.0 ** -8 * (6 + few.float().abs())).all())
    assert bool((lse[:, -8:] - fl).abs().max() <= 1e-4)
    assert bool(out.float().abs().sum(-1).gt(0).all())


def test_serving_loop(b):
    """append -> attend -> weights -> evict, as a decoder runs them, against the
    formulas over the rows that the cache holds at each step."""
    import torch
    outer, kvh, G, C, block, budget, window = 4, 2, 4, 128, 64, 5, 2
    cap, R = block * (budget + 2), 32
    kqo, vqo = S.formats()
    kqp, vqp = (b.QParams.asym(4, 0, 15, axis=a, group=64, residual=R, scale_dtype=b.BF16, zero_dtype=b.BF16)
                for a in (b.ALONG_T, b.ALONG_C))
    shape = (outer, cap, C)
    bufs = []
    for qp in (kqp, vqp):
        sizes = b.kvq_quantized_sizes(shape, b.BF16, b.QParams.asym(4, 0, 15, axis=qp.axis, group=64, scale_dtype=b.BF16,
                                                                      zero_dtype=b.BF16))
        bufs.append([torch.zeros(s, dtype=torch.uint8, device="cuda") for s in sizes[:3]] +
                    [torch.zeros((outer, R + block, C), dtype=torch.bfloat16, device="cuda")])
    ws = torch.empty(b.kvq_append_kv_workspace(shape, b.BF16, kqp, vqp, block), dtype=torch.uint8, device="cuda")
    app = b.KVAppender(shape, b.BF16, kqp, vqp, block, bufs[0], bufs[1], ws)
    cache = b.KVCache(k=tuple(bufs[0]), v=tuple(bufs[1]), shape=shape, kqp=kqp, vqp=vqp, tq=0, nres=0,
                      resid_rows=R + block, kv_heads=kvh)
    scores = torch.zeros((outer, cap + R + block), device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(11)

    def held():
        torch.cuda.synchronize()
        rows = []
        for bf, qo, mr in ((bufs[0], kqo, cache.tq // 64), (bufs[1], vqo, cache.tq)):
            x = np.zeros((outer, 0, C))
            if cache.tq:
                full = cap // 64 if qo is kqo else cap
                width = C if qo is kqo else C // 64
                codes = bf[0].cpu().numpy().reshape(outer, cap, C // 2)[:, :cache.tq]
                sc, ze = (S.bf16_to_f64(t.cpu().numpy().view(np.uint16).reshape(outer, full, width)[:, :mr]) for t in bf[1:3])
                c = np.stack([codes & 15, codes >> 4], -1).reshape(outer, cache.tq, C).astype(np.float64)
                rep = (1, 64) if qo is kqo else (2, 64)
                x = (c - np.repeat(ze, rep[1], rep[0])) * np.repeat(sc, rep[1], rep[0])
                x = S.bf16_to_f64(S.W.to_bf16_bits(x.astype(np.float32)))
            r = bf[3][:, :cache.nres].cpu().view(torch.int16).numpy().view(np.uint16)
            rows.append(np.concatenate([x, S.bf16_to_f64(r)], 1))
        return rows

    evictions = 0
    for step in range(150):
        n = 200 if step == 0 else 1 if step % 9 else 37       # a prompt, then tokens and drafted runs
        k, v = (torch.randn((outer, n, C), generator=gen, device="cuda").bfloat16() for _ in range(2))
        app.append(k, v, n)
        cache.tq, cache.nres = app.tq, app.nres
        q = (2 * torch.randn((outer // kvh, n, kvh * G, C), generator=gen, device="cuda")).bfloat16()
        out, lse = b.attend_chunk(q, cache)
        before = scores.clone()
        b.attend_weights(q, lse, cache, scores, scores)
        K, V = held()
        x, mag = S.logits(q.float().cpu().numpy().astype(np.float64), K, None, kvh)
        p, wl = S.softmax(x)
        e = 2 * S.logit_error(mag, x, C)
        u = 2.0 ** -8
        want, absout = np.einsum("oijt,otc->oijc", p, V), np.einsum("oijt,otc->oijc", p, np.abs(V))
        to = S.to_rows((u + e[..., None] + (cache.T + 64) * 2.0 ** -23) * absout, kvh) + u * np.abs(S.to_rows(want, kvh)) + 1e-30
        assert np.all(np.abs(out.float().cpu().numpy() - S.to_rows(want, kvh)) <= to), step
        # the weights use the kernel's own lse, off by at most e more than its rounding
        tw = np.einsum("oijt,oij->ot", p, 2 * e + (n * G + cache.T + 128) * 2.0 ** -23 + 16 * 2.0 ** -23 * (np.abs(wl) + 1))
        old = before[:, :cache.T].cpu().numpy().astype(np.float64)
        got = scores[:, :cache.T].cpu().numpy().astype(np.float64)
        assert np.all(np.abs(got - old - p.sum((1, 2))) <= tw + 2.0 ** -23 * (old + 1)), step
        if cache.tq > block * budget:
            nb, sc = cache.tq // block, scores.cpu().numpy()
            b.evict_blocks(cache, scores, budget, window, block)
            app.set_counters(cache.tq, cache.nres)
            K2, V2 = held()
            for o in range(outer):
                s = [sc[o, i * block:(i + 1) * block].astype(np.float64).sum() for i in range(nb - window)]
                ids = sorted(sorted(range(nb - window), key=lambda i: (-s[i], i))[:budget - window] + list(range(nb - window, nb)))
                tok = np.array([i * block + y for i in ids for y in range(block)] + list(range(nb * block, nb * block + cache.nres)))
                assert np.array_equal(K2[o], K[o, tok]) and np.array_equal(V2[o], V[o, tok])
                new = scores[o].cpu().numpy()
                assert np.array_equal(new[:len(tok)], sc[o, tok]) and not new[len(tok):].any()
            evictions += 1
    assert evictions >= 2 and cache.tq <= block * (budget + 1)
