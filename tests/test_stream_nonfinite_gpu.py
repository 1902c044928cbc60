"""kvq_attend_chunk and kvq_attend_weights where tokens hold NaN or infinities.

The definition sums over the tokens a query sees, so:
  * a logit that is NaN or +inf, seen, makes the row's out and lse NaN, and the
    weights of every token that the row sees; a logit of -inf is a weight of 0;
  * a value that is not finite reaches its channel of every row that sees its
    token (+inf, -inf, or NaN where both or a NaN are seen), and no other row;
  * rows that give nothing (lse = -inf) and rows that do not exist add nothing.
Whether a number is finite, and which infinity it is, is compared exactly; the
finite ones with the tolerances of test_stream_attend_gpu.py (u = 2^-8, the
largest relative error of a rounding to bf16; e twice the logits' error):
  lse: e + (T + 64) 2^-23 + 4 2^-23 (|lse| + 1)
  out: (u + e + (T + 64) 2^-23) sum_t p_t |v_t| + u |out|
  weights: (e + (rows + 64) 2^-23 + 8 2^-23 |lse|) sum w + 2^-23 sum w
"""
import zlib

import numpy as np
import pytest

import oracle as O
import stream_util as S
from gpu_util import kb

pytestmark = pytest.mark.gpu
NAN, INF = np.uint16(0x7FC0), np.uint16(0x7F80)
NEG = np.uint16(0xFF80)


@pytest.fixture(scope="module")
def b():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return kb()


# one case for each way through the kernels: batch, kv_heads, group, n, C, tq, cap, nres, rows, formats, first
FORMS = {
    "one token, one split": (2, 70, 4, 1, 128, 64, 64, 9, 16, {}, None),
    "one token, cluster": (1, 2, 4, 1, 128, 960, 1024, 40, 64, {}, None),
    "one token, workspace": (1, 2, 4, 1, 128, 9024, 9088, 40, 64, {}, None),
    "eight rows, two bits": (1, 2, 4, 2, 64, 448, 512, 1, 64, dict(bits=2, kind="sym", gv=32), None),
    "sixteen rows, padded": (3, 1, 4, 4, 128, 512, 576, 2, 64, {}, [0, 100, 511]),
    "twelve rows, cluster": (1, 1, 3, 4, 128, 1024, 1024, 2, 64, dict(kind="signed", gv=128), None),
    "32 rows, split": (1, 1, 8, 4, 128, 4096, 4096, 2, 64, dict(gv=32), None),
    "32 rows, symmetric": (1, 2, 8, 4, 64, 512, 512, 3, 64, dict(kind="sym", gk=128), None),
    "80 rows": (2, 1, 4, 20, 128, 512, 576, 7, 64, {}, [0, 130]),
    "160 rows, split": (1, 1, 8, 20, 128, 4096, 4096, 7, 192, {}, None),
    "240 rows, two bits": (1, 2, 8, 30, 64, 512, 576, 7, 64, dict(bits=2, gv=32), None),
    "520 rows": (1, 2, 4, 130, 64, 256, 256, 30, 64, dict(kind="sym"), None),
    "520 rows, split": (2, 1, 4, 130, 128, 2048, 2112, 45, 192, {}, [0, 300]),
    "520 rows, two bits": (1, 1, 4, 130, 128, 448, 448, 30, 64, dict(bits=2, gv=128), None),
}


def rows_of(c, oq, tq, nres):
    """The rows that raw buffers (codes, scale, zero, resid) stand for, binary64 [outer, T, C]."""
    import torch
    codes, sc, ze, r = c
    per = 8 // oq.bits
    C = r.shape[-1]
    x = np.stack([(codes[:, :tq] >> (oq.bits * k)) & ((1 << oq.bits) - 1) for k in range(per)], -1).astype(np.int32)
    x = x.reshape(codes.shape[0], tq, C)
    if oq.mode == O.SYM or oq.qmin < 0:
        x = (x ^ (1 << (oq.bits - 1))) - (1 << (oq.bits - 1))
    x = x.astype(np.float32)

    def spread(m):
        m = S.bf16_to_f64(m).astype(np.float32)
        if oq.axis == O.ALONG_T:
            return m[:, np.arange(tq) // oq.group]
        return m[:, :tq][:, :, np.arange(C) // (oq.group or C)]
    with np.errstate(invalid="ignore", over="ignore"):
        if ze is not None:
            x = x - spread(ze)
        x = x * spread(sc)
    x = torch.from_numpy(x).bfloat16().double().numpy()
    return np.concatenate([x, S.bf16_to_f64(r[:, :nres])], 1)


class Case:
    def __init__(self, name, what):
        self.B, self.H, self.G, self.n, self.C, tq, cap, nres, rows, fm, self.first = FORMS[name]
        rng = np.random.default_rng(zlib.crc32((name + what).encode()))
        self.hc = S.HostCache(rng, self.B * self.H, self.C, tq, cap, nres, rows, *S.formats(**{"gv": 64, **fm}))
        self.q = S.W.to_bf16_bits(rng.standard_normal((self.B, self.n, self.H * self.G, self.C)).astype(np.float32))
        POKE[what](self)
        hc = self.hc
        hc.K, hc.V = (rows_of(c, p, hc.tq, hc.nres) for c, p in ((hc.k, hc.kq), (hc.v, hc.vq)))
        T = hc.T
        f = np.zeros(hc.outer, np.int64) if self.first is None else np.asarray(self.first)
        self.seen = (np.arange(T) >= f[:, None, None]) & (np.arange(T) <= T - self.n + np.arange(self.n)[:, None])  # [o, i, t]

    def queries(self):
        import torch
        return torch.from_numpy(self.q.view(np.int16).copy()).view(torch.bfloat16).cuda()


def key_inf(c, negative):
    """+inf in channel 3 of buffered keys: logits are the sign of q's channel 3."""
    c.hc.k[3][:, c.hc.nres - 1, 3] = INF
    c.hc.k[3][:, 0, 3] = INF
    if negative:
        c.q[..., 3] |= 0x8000
    c.q[..., 3] |= 0x0080                                  # not zero


def q_nan(c):
    c.q[0, c.n // 2, 0, 5] = NAN


def q_inf(c):
    c.q[-1, c.n - 1, -1, 7] = NEG


def q_all(c):
    c.q[...] = NAN


def k_row(c):
    c.hc.k[3][0, c.hc.nres // 2, 1] = NAN


def k_group(c):
    """a key group's scale, so every logit of its tokens; slice 0 only"""
    c.hc.k[1][0, (c.hc.tq - 1) // c.hc.kq.group, 2] = NAN


def v_buffer(c):
    v, last = c.hc.v[3], c.hc.nres - 1
    v[:, last, 1], v[:, last, 2], v[:, last, 33] = INF, NEG, NAN
    v[0, 0, 5] = INF
    v[0, last, 5] = NEG                                    # rows that see both: NaN


def v_scale(bits):
    def poke(c):
        c.hc.v[1][0, c.hc.tq - 1, 0] = bits                # the newest store token, one group of channels
    return poke


def v_zero(c):
    if c.hc.v[2] is None:
        return v_scale(INF)(c)
    c.hc.v[2][0, c.hc.tq - 1, -1] = NEG


def far(c):
    """far zero points everywhere, and one value scale that is not finite"""
    for x in (c.hc.k, c.hc.v):
        if x[2] is not None:
            x[2][:, :] = S.W.to_bf16_bits(S.bf16_to_f64(x[2]).astype(np.float32) + 150)
    v_scale(INF)(c)


def far_scale(c):
    """scales beyond the bf16 route's, with finite values"""
    if c.hc.v[1] is not None:
        c.hc.v[1][0, c.hc.tq - 1] = S.W.to_bf16_bits(np.float32([3e35]))[0]
    v_buffer(c)


POKE = {"q nan": q_nan, "q inf": q_inf, "q all nan": q_all, "k row": k_row, "k group": k_group,
        "k inf": lambda c: key_inf(c, False), "k inf, away": lambda c: key_inf(c, True),
        "v buffer": v_buffer, "v scale inf": v_scale(INF), "v scale nan": v_scale(NAN), "v zero": v_zero,
        "far": far, "far scale": far_scale}
LOGITS = ["q nan", "q inf", "q all nan", "k row", "k group", "k inf", "k inf, away"]
VALUES = ["v buffer", "v scale inf", "v scale nan", "v zero", "far", "far scale"]


def solve(c):
    """x [o, i, j, t], mag, p, lse, poisoned [o, i, j]: rows with a NaN or +inf logit."""
    hc, q = c.hc, S.bf16_to_f64(c.q)
    with np.errstate(invalid="ignore"):
        x, mag = S.logits(q, hc.K, c.first, c.H)
        bad = (np.isnan(x) | (x == np.inf)).any(-1)
        x0 = np.where(bad[..., None], 0.0, x)               # such rows are not compared further
        p, lse = S.softmax(np.where(c.seen[:, :, None], x0, -np.inf))
    mag = np.where(np.isfinite(mag), mag, 0.0)              # a logit of -inf has no error
    return x0, mag, p, lse, bad


def check_out(c, got, gl):
    hc = c.hc
    x, mag, p, lse, bad = solve(c)
    V = np.where(np.isfinite(hc.V), hc.V, 0.0)
    out, absout = np.einsum("oijt,otc->oijc", p, V), np.einsum("oijt,otc->oijc", p, np.abs(V))
    seen = c.seen.astype(np.float64)
    plus = np.einsum("oit,otc->oic", seen, ((hc.V == np.inf) | np.isnan(hc.V)).astype(np.float64)) > 0
    minus = np.einsum("oit,otc->oic", seen, ((hc.V == -np.inf) | np.isnan(hc.V)).astype(np.float64)) > 0
    with np.errstate(invalid="ignore"):
        out = out + np.where(plus, np.inf, 0.0)[:, :, None] + np.where(minus, -np.inf, 0.0)[:, :, None]
    out = np.where(bad[..., None], np.nan, out)
    e = 2 * S.logit_error(mag, np.where(np.isfinite(x), x, 0.0), c.C)
    want, wl = S.to_rows(out, c.H), S.to_rows(np.where(bad, np.nan, lse), c.H)
    assert np.array_equal(np.isnan(gl), np.isnan(wl)), "lse: NaN"
    assert np.array_equal(np.isinf(gl), np.isinf(wl)), "lse: infinities"
    ok = np.isfinite(wl)
    tl = S.to_rows(e, c.H) + (hc.T + 64) * 2.0 ** -23 + 4 * 2.0 ** -23 * (np.abs(np.where(ok, wl, 0)) + 1)
    assert np.all(np.abs(gl[ok] - wl[ok]) <= tl[ok])
    assert np.array_equal(np.isnan(got), np.isnan(want)), "out: NaN"
    assert np.array_equal(np.isposinf(got), np.isposinf(want)) and np.array_equal(np.isneginf(got), np.isneginf(want))
    ok = np.isfinite(want)
    u = 2.0 ** -8
    to = S.to_rows((u + e[..., None] + (hc.T + 64) * 2.0 ** -23) * absout, c.H) + u * np.abs(np.where(ok, want, 0)) + 1e-30
    assert np.all(np.abs(got[ok] - want[ok]) <= to[ok])


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


@pytest.mark.parametrize("what", LOGITS)
@pytest.mark.parametrize("name", FORMS)
def test_logits_that_are_not_finite(b, name, what):
    c = Case(name, what)
    out, lse = b.attend_chunk(c.queries(), c.hc.device(b, c.H, c.first))
    check_out(c, host(out), host(lse))


@pytest.mark.parametrize("what", VALUES)
@pytest.mark.parametrize("name", FORMS)
def test_values_that_are_not_finite(b, name, what):
    c = Case(name, what)
    assert not np.isfinite(c.hc.V).all()
    out, lse = b.attend_chunk(c.queries(), c.hc.device(b, c.H, c.first))
    check_out(c, host(out), host(lse))


@pytest.mark.parametrize("what", LOGITS)
@pytest.mark.parametrize("name", FORMS)
def test_weights_of_logits_that_are_not_finite(b, name, what):
    """attend's lse into the weights: a poisoned row is not dropped, and nothing else is touched."""
    c = Case(name, what)
    cache, q = c.hc.device(b, c.H, c.first), c.queries()
    _, lse = b.attend_chunk(q, cache)
    got = host(b.attend_weights(q, lse, cache))
    x, mag, p, l64, bad = solve(c)
    nan = (bad.any(2)[:, :, None] & c.seen).any(1)           # [o, t]
    assert np.array_equal(np.isnan(got), nan)
    p = np.where(bad[..., None], 0.0, p)
    # lse is the kernel's own: off by at most e and its rounding, once more
    e = 2 * S.logit_error(mag, np.where(np.isfinite(x), x, 0.0), c.C)
    big = np.where(np.isfinite(l64), np.abs(l64), 0.0)
    tol = np.einsum("oijt,oij->ot", p, 2 * e + (c.n * c.G + c.hc.T + 128) * 2.0 ** -23 + 16 * 2.0 ** -23 * (big + 1)) + 1e-30
    w = p.sum((1, 2))
    assert np.all(np.abs(got - w)[~nan] <= tol[~nan])


@pytest.mark.parametrize("name", FORMS)
def test_rows_without_lse_give_nothing(b, name):
    """lse = -inf drops a row, whatever its query holds."""
    c = Case(name, "q nan")
    q, cache = c.queries(), c.hc.device(b, c.H, c.first)
    zero = q.clone()
    zero[0, c.n // 2, 0] = 0
    _, lse = b.attend_chunk(zero, cache)
    lse[0, c.n // 2, 0] = -float("inf")
    got, want = b.attend_weights(q, lse, cache), b.attend_weights(zero, lse, cache)
    assert bool(got.isfinite().all()) and np.array_equal(host(got), host(want))
