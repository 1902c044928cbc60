"""kvq_attend_shared against the formula in binary64: softmax over the prefix's
tokens and the requests' own.

Tolerances (u = 2^-8, the largest relative error of a rounding to bf16; e twice
the logits' error, stream_util.logit_error, the larger of the two parts'; T the
tokens of both):
  lse: e + (T + 128) 2^-23 + 12 2^-23 (|lse| + 1)
  out: (u + e + (T + 128) 2^-23 + 12 2^-23 (|lse| + 1)) sum_t p_t |v_t| + u |out|
A part's maximum in base 2 and its difference to the joined one are float32
numbers of the size of lse: a few more 2^-23 of it in the exponent than one
launch has.  Own results given as (out, lse) are one more token of that logit and
value, exact.
"""
import zlib

import numpy as np
import pytest

import serve_util as P
import stream_util as S
from gpu_util import Guarded, kb

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def b():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return kb()


#  batch, kv_heads, group, n, C, prefix (tq, nres, formats), own (tq, nres, formats) or "joined" or None, extras
CASES = {
    "one token of each": (1, 1, 1, 1, 128, (0, 1, {}), (0, 1, {}), {}),
    "one request": (1, 2, 4, 1, 128, (256, 30, {}), (64, 9, {}), {}),
    "few requests": (4, 2, 4, 1, 128, (832, 168, {}), (0, 90, {}), dict(first=[0, 10, 33, 89])),
    "eight rows a prefix": (2, 3, 4, 1, 64, (320, 40, dict(gv=32)), (128, 66, {}), {}),
    "32 rows": (8, 1, 4, 1, 128, (640, 77, {}), (192, 130, {}), dict(first=[0, 5, 64, 100, 191, 192, 321, 322])),
    "33 rows": (11, 1, 3, 1, 128, (640, 77, {}), (0, 30, {}), {}),
    "200 rows": (25, 2, 8, 1, 128, (1024, 100, {}), (64, 70, {}), dict(ragged=True)),
    "256 rows, C 64": (64, 1, 4, 1, 64, (448, 3, {}), (64, 11, dict(gv=32)), dict(ragged=True)),
    "600 rows": (75, 2, 8, 1, 128, (1088, 100, {}), (0, 20, {}), dict(ragged=True)),
    "600 rows, C 64": (75, 1, 8, 1, 64, (1088, 100, dict(gv=32)), (64, 20, {}), dict(ragged=True)),
    "drafts, two bits": (5, 2, 4, 5, 128, (960, 66, dict(bits=2, kind="sym", gk=32)), (128, 40, dict(bits=2, gk=32, gv=32)), {}),
    "bits that differ": (6, 1, 8, 1, 128, (512, 20, dict(bits=2, gk=32)), (64, 40, {}), {}),
    "chunks": (2, 2, 4, 70, 128, (512, 30, {}), (128, 72, {}), dict(first=[0, 0, 90, 150])),
    "chunks, C 64": (3, 1, 2, 150, 64, (256, 30, {}), (256, 0, {}), {}),
    "more queries than own tokens": (3, 1, 4, 9, 128, (256, 0, {}), (0, 4, {}), {}),
    "no own tokens": (3, 2, 4, 1, 128, (256, 5, {}), (0, 0, {}), {}),
    "empty prefix": (3, 2, 4, 2, 128, (0, 0, {}), (64, 5, {}), {}),
    "empty prefix, many rows": (30, 1, 4, 3, 128, (0, 0, {}), (64, 5, {}), {}),
    "nothing at all": (2, 1, 4, 1, 64, (0, 0, {}), (0, 0, {}), {}),
    "prefix alone": (5, 2, 8, 1, 128, (512, 40, {}), None, {}),
    "prefix alone, many rows": (5, 1, 8, 20, 128, (512, 40, {}), None, {}),
    "joined": (4, 2, 4, 1, 128, (512, 40, {}), "joined", {}),
    "joined, 200 rows": (1, 2, 4, 50, 128, (512, 40, {}), "joined", {}),
    "joined, prompts": (1, 2, 4, 333, 128, (640, 40, {}), "joined", {}),
    "joined, prompts, C 64": (1, 1, 3, 400, 64, (384, 1, {}), "joined", {}),
    "joined, empty prefix": (2, 1, 4, 1, 128, (0, 0, {}), "joined", {}),
    "long, split": (3, 1, 4, 1, 128, (9024, 100, {}), (64, 30, {}), {}),
    "long, split, 160 rows": (20, 1, 8, 1, 128, (4096, 100, {}), (64, 30, {}), {}),
    "far zero points": (12, 1, 4, 1, 128, (256, 20, {}), (64, 20, {}), dict(shift=100.0)),
    "padded prefix": (12, 2, 4, 1, 128, (256, 20, {}), (64, 20, {}), dict(pfirst=[100, 270])),
    "hidden prefix": (12, 2, 4, 1, 128, (256, 20, {}), (64, 20, {}), dict(pfirst=[999, 0])),
    "own tokens split too": (2, 1, 4, 1, 128, (512, 0, {}), (5056, 40, {}), {}),
    # the forms that pairs of SMs read: groups, kinds and ends of a prefix
    "pairs, key groups of 32": (20, 1, 8, 1, 128, (672, 9, dict(gk=32, gv=32)), (0, 9, {}), {}),
    "pairs, key groups of 96": (20, 2, 8, 1, 128, (960, 0, dict(gk=96, gv=128)), (0, 9, {}), {}),
    "pairs, key groups of 128, symmetric": (20, 1, 8, 1, 128, (896, 70, dict(gk=128, kind="sym")), (64, 9, {}), {}),
    "pairs, signed": (20, 1, 8, 1, 128, (512, 129, dict(kind="signed", gv=32)), (0, 9, {}), {}),
    "pairs, two bits": (40, 1, 8, 1, 128, (448, 1, dict(bits=2, gk=64, gv=128)), (64, 9, {}), dict(ragged=True)),
    "pairs, two bits, symmetric": (70, 1, 8, 1, 128, (704, 33, dict(bits=2, kind="sym", gk=32, gv=32)), (0, 9, {}), {}),
    "pairs, one tile": (20, 1, 8, 1, 128, (64, 30, {}), (0, 9, {}), {}),
    "pairs, buffer only": (20, 1, 8, 1, 128, (0, 61, {}), (0, 9, {}), {}),
    "pairs, padded": (20, 3, 4, 1, 128, (640, 60, {}), (0, 9, {}), dict(pfirst=[64, 130, 655])),
    "pairs, hidden": (40, 2, 4, 1, 128, (640, 60, {}), (0, 9, {}), dict(pfirst=[700, 699])),
    "pairs, far zero points": (40, 1, 4, 1, 128, (512, 20, {}), (0, 9, {}), dict(shift=100.0)),
    "pairs, 257 rows": (257, 1, 1, 1, 128, (256, 20, {}), (0, 3, {}), {}),
    "pairs, 2000 rows, split": (250, 1, 8, 1, 128, (2048, 100, {}), (0, 9, {}), dict(ragged=True)),
    # 33 to 128 rows
    "one tile, 33 rows": (11, 1, 3, 1, 128, (64, 30, {}), (0, 9, {}), {}),
    "two bits, 80 rows": (10, 1, 8, 1, 128, (448, 1, dict(bits=2, gk=64, gv=128)), (64, 9, {}), dict(ragged=True)),
    "key groups of 96, 128 rows": (16, 2, 8, 1, 128, (960, 0, dict(gk=96, gv=128)), (0, 9, {}), {}),
    "129 rows": (129, 1, 1, 1, 128, (512, 129, dict(kind="signed", gv=32)), (0, 9, {}), {}),
    "joined, 100 rows": (1, 2, 4, 25, 128, (512, 40, {}), "joined", {}),
    "2100 rows": (300, 1, 7, 1, 128, (512, 100, {}), (0, 9, {}), {}),
    "2100 rows of chunks": (6, 1, 7, 50, 128, (512, 100, {}), (64, 20, {}), dict(first=[0, 80, 33, 1, 84, 20])),
    "2100 rows, split": (1, 1, 7, 300, 128, (4096, 100, {}), "joined", {}),
}


def build(name):
    rng = np.random.default_rng(zlib.crc32(name.encode()))
    B, H, G, n, C, pre, own, ex = CASES[name]

    def cache(outer, spec):
        tq, nres, fm = spec
        gk = fm.get("gk", 64)
        return S.HostCache(rng, outer, C, tq, tq + gk, nres, nres + gk, *S.formats(**{"gv": 64, **fm}), ex.get("shift", 0.0))

    prefix = cache(H, pre)
    mine = cache(B * H, own) if isinstance(own, tuple) else own
    first = ex.get("first")
    if first and len(first) == B:
        first = [f for f in first for _ in range(H)]
    if ex.get("ragged"):
        first = [int(v) for v in rng.integers(0, mine.T + 1, B) for _ in range(H)]
    q = S.W.to_bf16_bits(rng.standard_normal((B, n, H * G, C)).astype(np.float32))
    if own == "joined":
        y = S.W.to_bf16_bits(rng.standard_normal((B, n, H * G, C)).astype(np.float32))
        z = (5.0 + rng.standard_normal((B, n, H * G))).astype(np.float32)
        z[0, 0, 0] = -np.inf                     # saw nothing, whatever its out holds
        y[0, 0, 0] = 0x7FC0
        mine = (y, z)
    return prefix, mine, q, first


def hide(hc, first):
    K, V = hc.K.copy(), hc.V.copy()
    for o, f in enumerate(first if first is not None else []):
        K[o, :max(f, 0)] = V[o, :max(f, 0)] = 0.0
    return K, V


def reference(name, prefix, mine, q, first):
    B, H, G, n, C, _, _, ex = CASES[name]
    qd = S.bf16_to_f64(q)
    K, V = hide(prefix, ex.get("pfirst"))
    # every query sees the whole prefix: n = 1, one row for each query and head of a KV head
    rows = qd.reshape(B * n, H, G, C).transpose(1, 0, 2, 3).reshape(1, 1, H * B * n * G, C)
    x, mag = S.logits(rows, K, ex.get("pfirst"), H)

    def back(t):
        return t.reshape(H, B, n, G, -1).transpose(1, 2, 0, 3, 4).reshape(B, n, H * G, -1)

    xs, mags = [back(x)], [back(mag)]
    vals = [np.broadcast_to(np.repeat(V, G, 0)[None, None], (B, n, H * G, *V.shape[1:]))]
    if isinstance(mine, S.HostCache):
        K, V = hide(mine, first)
        x, mag = S.logits(qd, K, first, H)
        xs.append(S.to_rows(x, H))
        mags.append(S.to_rows(mag, H))
        v = np.repeat(V.reshape(B, 1, H, -1, C), G, 2)
        vals.append(np.broadcast_to(v, (B, n, *v.shape[2:])))
    elif mine is not None:
        y, z = mine
        xs.append(z.astype(np.float64)[..., None])
        mags.append(np.zeros_like(xs[-1]))
        vals.append(np.where(np.isinf(xs[-1]), 0.0, S.bf16_to_f64(y))[..., None, :])
    x, mag = np.concatenate(xs, -1), np.concatenate(mags, -1)
    p, lse = S.softmax(x)
    out, absout, at = 0.0, 0.0, 0
    for v in vals:
        w = p[..., at:at + v.shape[-2]]
        out = out + np.einsum("bnht,bnhtc->bnhc", w, v)
        absout = absout + np.einsum("bnht,bnhtc->bnhc", w, np.abs(v))
        at += v.shape[-2]
    return lse, out, absout, 2.0 * S.logit_error(mag, x, C), x.shape[-1]


def tolerances(lse, out, absout, e, T):
    size = 12 * 2.0 ** -23 * (np.where(np.isfinite(lse), np.abs(lse), 0.0) + 1.0) + (T + 128) * 2.0 ** -23
    return e + size, (P.U + e + size)[..., None] * absout + P.U * np.abs(out)


def run(b, name, g=None):
    import torch
    prefix, mine, q, first = build(name)
    B, H, G, n, C, _, _, ex = CASES[name]
    pc = prefix.device(b, H, ex.get("pfirst"))
    cache = mine.device(b, H, first) if isinstance(mine, S.HostCache) else None
    own = (P.upload_bf16(mine[0]), torch.from_numpy(mine[1]).cuda()) if isinstance(mine, tuple) else None
    g = g or Guarded()
    out = g.alloc(q.size * 2).view(torch.bfloat16).view(q.shape)
    lse = g.alloc(q.size // C * 4).view(torch.float32).view(q.shape[:3])
    wB = b.kvq_attend_shared_workspace(pc.shape, pc.resid_rows, None if cache is None else cache.shape,
                                       0 if cache is None else cache.resid_rows, B, n, G)
    ws = g.alloc(max(wB, 16))
    return P.upload_bf16(q), pc, cache, own, out, lse, ws, g, reference(name, prefix, mine, q, first)


@pytest.mark.parametrize("name", CASES)
def test_attend_shared(b, name):
    q, pc, cache, own, out, lse, ws, g, ref = run(b, name)
    b.attend_shared(q, pc, cache, own, out, lse, ws)
    g.check(name)
    tl, to = tolerances(*ref)
    P.close(P.f64(lse), ref[0], tl, name + ": lse")
    P.close(P.f64(out), ref[1], to, name + ": out")


@pytest.mark.parametrize("name", ["few requests", "200 rows", "joined", "joined, prompts", "chunks"])
def test_in_place_and_default_arguments(b, name):
    import torch
    q, pc, cache, own, *_ = run(b, name)
    want = b.attend_shared(q, pc, cache, own)
    if own is None:
        y = q.clone()
        b.attend_shared(y, pc, cache, out=y)
        assert torch.equal(y, want[0])
    else:
        b.attend_shared(q, pc, own=own, out=own[0], lse=own[1])
        assert torch.equal(own[0], want[0]) and torch.equal(own[1], want[1])


@pytest.mark.parametrize("name", ["few requests", "32 rows", "200 rows", "600 rows", "chunks", "joined, prompts", "long, split",
                                  "pairs, two bits", "2100 rows of chunks"])
def test_captured_and_on_two_streams(b, name):
    """Two captured graphs with a workspace each, replayed on two streams, give the bits of an eager call."""
    import torch
    q, pc, cache, own, out, lse, ws, g, _ = run(b, name)
    want = b.attend_shared(q, pc, cache, own, workspace=ws)
    torch.cuda.synchronize()
    runs = []
    for _ in range(2):
        o, z, w = torch.empty_like(want[0]), torch.empty_like(want[1]), torch.empty_like(ws)
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            b.attend_shared(q, pc, cache, own, o, z, w)
        runs.append((gr, o, z, torch.cuda.Stream()))
    for _ in range(3):
        for gr, o, z, st in runs:
            with torch.cuda.stream(st):
                o.zero_()
                gr.replay()
    torch.cuda.synchronize()
    for _, o, z, _ in runs:
        assert torch.equal(o, want[0]) and torch.equal(z, want[1])


def test_values_that_are_not_finite(b):
    """An infinity in the prefix reaches its channel of every row, one of a request only that request's rows that see it."""
    import torch
    for B, n in ((3, 2), (40, 2), (150, 2)):                            # each form of the prefix's launch
        rng = np.random.default_rng(B)
        H, G, C = 1, 2, 128
        kq, vq = S.formats(gv=64)
        pre, mine = S.HostCache(rng, H, C, 256, 256, 20, 64, kq, vq), S.HostCache(rng, B * H, C, 64, 64, 12, 64, kq, vq)
        pre.v[3][0, 4, 7] = 0x7F80               # buffer row
        mine.v[3][1, 11, 9] = 0xFF80             # request 1's newest token: its last query sees it
        q = P.upload_bf16(S.W.to_bf16_bits(rng.standard_normal((B, n, H * G, C)).astype(np.float32)))
        out, lse = b.attend_shared(q, pre.device(b, H), mine.device(b, H))
        assert torch.isfinite(lse).all()
        assert (out[..., 7] == float("inf")).all()
        assert (out[1, 1, :, 9] == -float("inf")).all()
        ok = torch.ones_like(out, dtype=torch.bool)
        ok[..., 7] = False
        ok[1, 1, :, 9] = False
        assert torch.isfinite(out[ok]).all()


def test_stored_values_that_are_not_finite(b):
    """Scales of the prefix's values that are infinite or NaN: every channel of their group, in every row, whichever of
    a pair's SMs has the channels; and NaN in hidden tokens reaches nothing."""
    import torch
    for B in (3, 40, 300):
        rng = np.random.default_rng(B)
        H, G, C = 1, 8, 128
        pre = S.HostCache(rng, H, C, 512, 512, 20, 64, *S.formats(gv=32))
        q = P.upload_bf16(S.W.to_bf16_bits(rng.standard_normal((B, 1, H * G, C)).astype(np.float32)))
        pre.v[1][0, :100] = 0x7FC0               # padding
        pre.v[3][0, 20:] = 0x7FC0                # behind the filled rows
        want = b.attend_shared(q, pre.device(b, H, [100]))
        assert torch.isfinite(want[0]).all() and torch.isfinite(want[1]).all()
        pre.v[1][0, 300, 1] = 0x7FC0             # channels 32 .. 63 of a token
        pre.v[1][0, 433, 3] = 0x7FC0             # channels 96 .. 127 of one in another half tile
        out, lse = b.attend_shared(q, pre.device(b, H, [100]))
        assert torch.equal(lse, want[1])
        nan = torch.zeros(C, dtype=torch.bool, device="cuda")
        nan[32:64] = nan[96:] = True
        assert out[..., nan].isnan().all() and torch.equal(out[..., ~nan], want[0][..., ~nan])


def test_keys_that_are_nan(b):
    """A prefix key of NaN makes NaN of the KV head that has it, whatever the own tokens say, and of no other."""
    import torch
    for B in (3, 40, 300):
        rng = np.random.default_rng(B)
        H, G, C = 2, 8, 128
        pre = S.HostCache(rng, H, C, 256, 256, 20, 64, *S.formats())
        own = S.HostCache(rng, B * H, C, 0, 64, 9, 64, *S.formats())
        pre.k[3][1, 7, 5] = 0x7FC0
        q = P.upload_bf16(S.W.to_bf16_bits(rng.standard_normal((B, 1, H * G, C)).astype(np.float32)))
        out, lse = b.attend_shared(q, pre.device(b, H), own.device(b, H))
        assert torch.isfinite(out[:, :, :G]).all() and torch.isfinite(lse[:, :, :G]).all()
        assert out[:, :, G:].isnan().all() and lse[:, :, G:].isnan().all()


def test_rows_that_are_nan_stay_nan(b):
    import torch
    q, pc, cache, own, *_ = run(b, "joined")
    own[1][1, 0, 2] = float("nan")
    own[0][1, 0, 2] = float("nan")
    out, lse = b.attend_shared(q, pc, own=own)
    assert out[1, 0, 2].isnan().all() and lse[1, 0, 2].isnan()
    lse[1, 0, 2], out[1, 0, 2] = 0.0, 0.0
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()


def test_a_batch_from_prompts_to_tokens(b):
    """The three operators as a serving loop runs them: prompts behind a shared prefix, a cache filled from them, and
    decode steps over both, against attention over everything in binary64 (the quantized rows as they stand)."""
    import torch
    rng = np.random.default_rng(77)
    Hk, G, C, R, g = 2, 4, 128, 128, 64
    lens, H = [300, 41, 170], 8
    B, total, T = len(lens), sum(lens), max(lens)
    kq, vq = (b.QParams.asym(4, 0, 15, axis=a, group=64, residual=R, scale_dtype=b.BF16, zero_dtype=b.BF16)
              for a in (b.ALONG_T, b.ALONG_C))

    def empty(outer):
        sizes = [b._store_sizes((outer, 512, C), p, R + g) for p in (kq, vq)]
        return b.KVCache(*[tuple(torch.zeros(s, dtype=torch.uint8, device="cuda") for s in z) for z in sizes],
                         shape=(outer, 512, C), kqp=kq, vqp=vq, tq=0, nres=0, resid_rows=R + g, kv_heads=Hk)

    def rows(cache):
        """The bf16 rows of a cache's T tokens [outer, T, C], k and v."""
        found = []
        for bufs, p in ((cache.k, kq), (cache.v, vq)):
            st = b.QParams.asym(4, 0, 15, axis=p.axis, group=64, scale_dtype=b.BF16, zero_dtype=b.BF16)
            qt = b.Quantized(bufs[0], bufs[1], bufs[2], None, cache.shape, st, b.BF16)
            x = b.dequantize(qt)[:, :cache.tq]
            r = bufs[3].view(torch.bfloat16).view(cache.shape[0], R + g, C)[:, :cache.nres]
            found.append(P.f64(torch.cat([x, r], 1)))
        return found

    # the prefix: one prompt of its own
    px = P.upload_bf16(P.packed(rng, 391, H + 2 * Hk, C))
    one = torch.tensor([0, 391], dtype=torch.int32, device="cuda")
    prefix = b.fill_prompts(px[:, H:H + Hk], px[:, H + Hk:], one, empty(Hk), 391)
    # the prompts behind it
    x = P.packed(rng, total, H + 2 * Hk, C)
    dx, starts = P.upload_bf16(x), P.starts_of(lens)
    st = torch.from_numpy(starts).cuda()
    q, k, v = dx.split([H, Hk, Hk], 1)
    own = b.attend_prompts(q, k, v, st)
    y, z = b.attend_shared(q.contiguous()[None], prefix, own=(own[0][None], own[1][None]))
    PK, PV = rows(prefix)

    def expect(qr, K, V, h):                     # one query row over prefix and own rows of KV head h
        kk, vv = np.concatenate([PK[h], K]), np.concatenate([PV[h], V])
        lg = kk @ qr / np.sqrt(C)
        mag = np.abs(kk) @ np.abs(qr) / np.sqrt(C)
        p, lse = S.softmax(lg[None])
        return lse[0], (p @ vv)[0], (p @ np.abs(vv))[0], 2.0 * S.logit_error(mag[None], lg[None], C)[0], len(kk)

    def check(what, lse, out, args):
        wl, wo, wa, e, n = expect(*args)
        tl, to = tolerances(np.array(wl), wo, wa, np.array(e), n)
        # the prompts' own part has been rounded to bf16 once more than `tolerances` counts
        P.close(np.array(lse), np.array(wl), tl, what)
        P.close(out, wo, to + P.U * wa, what)

    xr = S.bf16_to_f64(x)
    gy, gz = P.f64(y[0]), P.f64(z[0])
    for s, n in enumerate(lens):
        for i in (0, n // 2, n - 1):
            for head in (0, 5):
                h, a = head // G, starts[s]
                check(f"prompt {s}, token {i}", gz[a + i, head], gy[a + i, head],
                      (xr[a + i, head], xr[a:a + i + 1, H + h], xr[a:a + i + 1, H + Hk + h], h))
    # into a cache, then decode steps across a flush of the buffer
    cache = b.fill_prompts(k, v, st, empty(B * Hk), T)
    ws = torch.empty(b.kvq_append_kv_workspace(cache.shape, b.BF16, kq, vq, g), dtype=torch.uint8, device="cuda")
    app = b.KVAppender(cache.shape, b.BF16, kq, vq, g, cache.k, cache.v, ws, cache.tq, cache.nres)
    for step in range(30):
        new = P.upload_bf16(P.packed(rng, B, H + 2 * Hk, C))
        app.append(new[:, H:H + Hk].reshape(B * Hk, 1, C).contiguous(), new[:, H + Hk:].reshape(B * Hk, 1, C).contiguous(), 1)
        cache.tq, cache.nres = app.tq, app.nres
        if step % 7:
            continue
        qn = new[:, None, :H].contiguous()
        y, z = b.attend_shared(qn, prefix, cache)
        K, V = rows(cache)
        gy, gz, gq = P.f64(y), P.f64(z), P.f64(qn)
        for s in range(B):
            for head in range(H):
                o = s * Hk + head // G
                f = T - lens[s]
                check(f"step {step}, request {s}", gz[s, 0, head], gy[s, 0, head],
                      (gq[s, 0, head], K[o, f:], V[o, f:], head // G))
    assert cache.tq > 128, "no flush happened"
