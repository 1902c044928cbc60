"""kvq_fill_prompts against the quantizer's definition, bit for bit: every group's
codes, scale and zero point are those of the oracle over the tokens that are
there, buffer rows are copies, and nothing else is written."""
import zlib

import numpy as np
import pytest

import oracle as O
import serve_util as P
import stream_util as S
from gpu_util import Guarded, kb, kq_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def b():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return kb()


#  lens, kv_heads, C, tq, nres, cap, rows, formats, extras
CASES = {
    "one token": ([1], 1, 128, 0, 1, 64, 64, {}, {}),
    "one token in the store": ([1], 1, 128, 64, 0, 64, 0, {}, {}),
    "one token of a group": ([65], 2, 128, 128, 0, 128, 0, {}, {}),
    "buffer only": ([100, 30], 2, 128, 0, 100, 64, 192, {}, {}),
    "store only": ([64, 128], 2, 128, 128, 0, 128, 0, {}, {}),
    "ragged": ([3, 700, 1, 64, 250, 511, 129, 0], 2, 128, 576, 124, 640, 192, {}, dict(fused=True)),
    "longer than the cache": ([500, 40], 2, 128, 128, 40, 192, 64, {}, {}),
    "shorter than the cache": ([5, 40], 2, 64, 128, 40, 192, 64, dict(gv=32), {}),
    "rows outside": ([40, 150], 2, 128, 64, 86, 64, 128, {}, dict(before=9, behind=5)),
    "two bits, symmetric": ([333, 90], 3, 128, 256, 77, 256, 96, dict(bits=2, kind="sym", gk=32, gv=32), dict(fused=True)),
    "two bits, C 64": ([200, 131], 2, 64, 128, 72, 160, 96, dict(bits=2, gk=32, gv=64), {}),
    "two bits, signed": ([150], 1, 128, 128, 22, 128, 64, dict(bits=2, kind="signed", gk=64, gv=128), {}),
    "symmetric, C 64": ([300, 140, 2], 2, 64, 256, 44, 256, 64, dict(kind="sym", gk=128, gv=64), {}),
    "signed zero points": ([300, 140], 2, 128, 256, 44, 256, 64, dict(kind="signed", gk=64, gv=128), {}),
    "groups of 96": ([500, 97], 2, 128, 384, 116, 480, 224, dict(gk=96), {}),
    "groups of 256": ([900, 300, 257], 1, 128, 768, 132, 1024, 384, dict(gk=256), {}),
    "groups of 1024, two bits": ([1200, 1030], 1, 64, 1024, 176, 1024, 200, dict(bits=2, gk=1024, gv=32), {}),
    "constant": ([200, 3], 1, 128, 128, 72, 128, 192, {}, dict(constant=True)),
    "tiny values": ([200, 70], 1, 128, 128, 72, 128, 192, {}, dict(scale=1e-36)),
    "far from zero": ([200, 70], 1, 128, 128, 72, 128, 192, {}, dict(shift=100.0)),
    "large values": ([200, 70], 1, 128, 128, 72, 128, 192, dict(kind="sym"), dict(scale=1e37)),
    "many prompts": ([(i * 53) % 170 for i in range(150)], 1, 64, 64, 100, 64, 128, {}, dict(fused=True)),
}


def build(name):
    rng = np.random.default_rng(zlib.crc32(name.encode()))
    lens, Hk, C, tq, nres, cap, rows, fm, ex = CASES[name]
    kq, vq = S.formats(**{"gv": 64, **fm})
    total = ex.get("before", 0) + sum(lens) + ex.get("behind", 0)
    x = rng.standard_normal((total, 2 * Hk, C)) * ex.get("scale", 1.0) + ex.get("shift", 0.0)
    if ex.get("constant"):
        x[:] = x[:1]
    return lens, Hk, C, tq, nres, cap, rows, kq, vq, ex, S.W.to_bf16_bits(x.astype(np.float32)), P.starts_of(lens, ex.get("before", 0))


def expected(name):
    """[k buffers, v buffers] as numpy, what is not written left as 0xA5 bytes, and first."""
    lens, Hk, C, tq, nres, cap, rows, kq, vq, _, x, starts = build(name)
    outer, T = len(lens) * Hk, tq + nres
    res, first = [], np.array([max(T - n, 0) for n in lens for _ in range(Hk)], np.int32)
    for oq, w in ((kq, 0), (vq, 1)):
        mr, mc = S.meta_rows(oq, cap, C)
        bufs = [np.full((outer, cap, C * oq.bits // 8), 0xA5, np.uint8), np.full((outer, mr, mc), 0xA5A5, np.uint16),
                None if oq.mode == O.SYM else np.full((outer, mr, mc), 0xA5A5, np.uint16),
                np.full((outer, rows, C), 0xA5A5, np.uint16)]
        for s, n in enumerate(lens):
            for h in range(Hk):
                o, f = s * Hk + h, max(T - n, 0)
                row = np.zeros((T, C), np.uint16)
                row[f:] = x[starts[s + 1] - (T - f):starts[s + 1], w * Hk + h]
                bufs[3][o, max(f - tq, 0):nres] = row[tq + max(f - tq, 0):]
                if oq.axis == O.ALONG_C:
                    pieces = [(f, tq)] if f < tq else []
                else:
                    pieces = [(max(a, f), a + oq.group) for a in range(0, tq, oq.group) if f < a + oq.group]
                for a, z in pieces:
                    one = O.QParams(oq.bits, oq.mode, oq.qmin, oq.qmax, oq.axis, 0 if oq.axis == O.ALONG_T else oq.group, 0,
                                    oq.scale_dtype, oq.zero_dtype)
                    qt = O.quantize(row[None, a:z], O.BF16, one)
                    bufs[0][o, a:z] = qt.codes.reshape(z - a, -1)
                    at = slice(a // oq.group, a // oq.group + 1) if oq.axis == O.ALONG_T else slice(a, z)
                    bufs[1][o, at] = qt.scale.reshape(-1, mc)
                    if bufs[2] is not None:
                        bufs[2][o, at] = qt.zero.reshape(-1, mc)
        res.append(bufs)
    return res, first


def device_cache(b, name, g):
    import torch
    lens, Hk, C, tq, nres, cap, rows, kq, vq, *_ = build(name)
    want, _ = expected(name)
    bufs = [tuple(None if a is None or a.nbytes == 0 else g.alloc(a.nbytes, fill=0xA5) for a in w) for w in want]
    first = g.alloc(len(lens) * Hk * 4).view(torch.int32)
    return b.KVCache(*bufs, shape=(len(lens) * Hk, cap, C), kqp=kq_of(b, kq), vqp=kq_of(b, vq), tq=tq, nres=nres,
                     resid_rows=rows, kv_heads=Hk, first=first)


def compare(name, cache):
    want, first = expected(name)
    assert np.array_equal(cache.first.cpu().numpy(), first), "first"
    for who, dev, host in zip("kv", (cache.k, cache.v), want):
        for part, d, h in zip(("codes", "scale", "zero", "resid"), dev, host):
            if d is None:
                continue
            got = d.cpu().numpy().view(h.dtype).reshape(h.shape)
            assert np.array_equal(got, h), f"{name}: {who} {part} differ first at {np.argwhere(got != h)[0]}"


def call(b, name, cache, stream=None):
    """The C entry point with the case's own counters."""
    import torch
    lens, Hk, C, *_, ex, x, starts = build(name)
    t = P.upload_bf16(x)
    k, v = t.split([Hk, Hk], 1)
    if not ex.get("fused"):
        k, v = k.contiguous(), v.contiguous()
    b.kvq_fill_prompts(k, k.stride(0), v, v.stride(0), torch.from_numpy(starts).cuda(), len(lens), x.shape[0], Hk, cache.c(),
                       cache.kqp, cache.vqp, cache.shape, stream)


@pytest.mark.parametrize("name", CASES)
def test_fill_prompts(b, name):
    g = Guarded()
    cache = device_cache(b, name, g)
    call(b, name, cache)
    g.check(name)
    compare(name, cache)


def test_a_cache_filled_from_one_length_equals_appends(b):
    """Prompts of one length: the same cache as appending their tokens, which a serving loop then goes on with."""
    import torch
    B, Hk, C, R, g, n = 2, 2, 128, 128, 64, 391
    rng = np.random.default_rng(3)
    x = P.upload_bf16(P.packed(rng, B * n, 2 * Hk, C))
    kw = dict(scale_dtype=b.BF16, zero_dtype=b.BF16, residual=R)
    kqp, vqp = (b.QParams.asym(4, 0, 15, axis=a, group=64, **kw) for a in (b.ALONG_T, b.ALONG_C))

    def empty():
        sizes = [b._store_sizes((B * Hk, 512, C), p, R + g) for p in (kqp, vqp)]
        bufs = [tuple(torch.zeros(s, dtype=torch.uint8, device="cuda") for s in z) for z in sizes]
        return b.KVCache(*bufs, shape=(B * Hk, 512, C), kqp=kqp, vqp=vqp, tq=0, nres=0, resid_rows=R + g, kv_heads=Hk)

    filled = b.fill_prompts(x[:, :Hk], x[:, Hk:], torch.from_numpy(P.starts_of([n] * B)).cuda(), empty(), n)
    other = empty()
    ws = torch.empty(b.kvq_append_kv_workspace(other.shape, b.BF16, kqp, vqp, g), dtype=torch.uint8, device="cuda")
    app = b.KVAppender(other.shape, b.BF16, kqp, vqp, g, other.k, other.v, ws)
    kv = x.view(B, n, 2, Hk, C).permute(2, 0, 3, 1, 4).reshape(2, B * Hk, n, C).contiguous()
    app.append(kv[0], kv[1], n)
    assert (filled.tq, filled.nres) == (app.tq, app.nres) and (filled.first == 0).all()
    for a, c in zip((*filled.k[:3], *filled.v[:3]), (*other.k[:3], *other.v[:3])):
        assert torch.equal(a, c)
    for a, c in ((filled.k[3], other.k[3]), (filled.v[3], other.v[3])):
        a, c = (t.view(torch.bfloat16).view(B * Hk, R + g, C)[:, :filled.nres] for t in (a, c))
        assert torch.equal(a, c)


def test_prompts_of_no_tokens(b):
    """Tensors without tokens, whatever their strides: a cache of padding alone."""
    import torch
    kw = dict(scale_dtype=b.BF16, zero_dtype=b.BF16, residual=64)
    kqp, vqp = (b.QParams.asym(4, 0, 15, axis=a, group=64, **kw) for a in (b.ALONG_T, b.ALONG_C))
    bufs = [tuple(torch.full((s,), 0xA5, dtype=torch.uint8, device="cuda") for s in b._store_sizes((2, 128, 64), p, 128))
            for p in (kqp, vqp)]
    cache = b.KVCache(*bufs, shape=(2, 128, 64), kqp=kqp, vqp=vqp, tq=0, nres=0, resid_rows=128, kv_heads=1)
    none = torch.empty(1, dtype=torch.bfloat16, device="cuda").as_strided((0, 1, 64), (0, 0, 0))
    b.fill_prompts(none, none, torch.zeros(3, dtype=torch.int32, device="cuda"), cache, 150)
    assert (cache.tq, cache.nres) == (64, 86) and (cache.first == 150).all()
    assert all((t == 0xA5).all() for t in (*cache.k, *cache.v))


def test_captured_fill_replays_with_other_lengths_and_streams(b):
    import torch
    name = "ragged"
    lens, Hk, C, *_, x, starts = build(name)
    g = Guarded()
    cache = device_cache(b, name, g)
    t = P.upload_bf16(x)
    st = torch.zeros(len(lens) + 1, dtype=torch.int32, device="cuda")
    args = (t[:, :Hk], t.stride(0), t[:, Hk:], t.stride(0), st, len(lens), x.shape[0], Hk, cache.c(), cache.kqp, cache.vqp,
            cache.shape)
    b.kvq_fill_prompts(*args)                    # no prompt has a token: all padding
    torch.cuda.synchronize()
    assert (cache.first == cache.T).all() and all((d == 0xA5).all() for d in (*cache.k, *cache.v))
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        b.kvq_fill_prompts(*args)
    st.copy_(torch.from_numpy(starts))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        gr.replay()
    g.check(name)
    compare(name, cache)


@pytest.mark.parametrize("starts", [[-5, 40, 1000], [30, 10, 60], [0, 2**31 - 1, 5], [-2**31, 2**31 - 1, 0], [60, 0, 0]])
def test_starts_out_of_order_or_range_stay_inside(b, starts):
    import torch
    Hk, C = 2, 128
    g = Guarded()
    x = P.upload_bf16(P.packed(np.random.default_rng(5), 60, 2 * Hk, C))
    kqp, vqp = (kq_of(b, p) for p in S.formats())
    sizes = [b._store_sizes((4, 64, C), p, 64) for p in (kqp, vqp)]
    cache = b.KVCache(*[tuple(g.alloc(s) for s in z) for z in sizes], shape=(4, 64, C), kqp=kqp, vqp=vqp, tq=64, nres=10,
                      resid_rows=64, kv_heads=Hk, first=g.alloc(16).view(torch.int32))
    st = torch.tensor(starts, dtype=torch.int64).to(torch.int32).cuda()
    b.kvq_fill_prompts(x[:, :Hk], x.stride(0), x[:, Hk:], x.stride(0), st, 2, 60, Hk, cache.c(), kqp, vqp, cache.shape)
    g.check("starts")
    assert ((cache.first >= 0) & (cache.first <= 74)).all()
