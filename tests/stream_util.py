"""Streaming caches for the tests of kvq_cache.h: built on the host by the
oracle's quantizer, uploaded into stores and buffers whose unused parts hold
NaN bit patterns, with the bf16 rows they stand for in binary64."""
import numpy as np

import oracle as O
from gpu_util import kq_of
from kv_cache_quantization_kvq_gb300 import workloads as W


def formats(bits=4, kind="asym", gk=64, gv=64):
    kw = dict(scale_dtype=O.BF16)
    if kind == "sym":
        return (O.QParams.sym(bits, axis=O.ALONG_T, group=gk, **kw), O.QParams.sym(bits, axis=O.ALONG_C, group=gv, **kw))
    lo, hi = (0, (1 << bits) - 1) if kind == "asym" else (-(1 << (bits - 1)), (1 << (bits - 1)) - 1)
    return tuple(O.QParams.asym(bits, lo, hi, axis=a, group=g, zero_dtype=O.BF16, **kw)
                 for a, g in ((O.ALONG_T, gk), (O.ALONG_C, gv)))


def bf16_to_f64(bits):
    return (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def meta_rows(oq, T, C):
    """(rows of the metadata's middle axis, row length)."""
    return (-(-T // oq.group), C) if oq.axis == O.ALONG_T else (T, -(-C // (oq.group or C)))


class HostCache:
    """k, v: (codes, scale, zero, resid) numpy arrays [outer, ...]; K, V: the
    rows in binary64 [outer, T, C]."""

    def __init__(self, rng, outer, C, tq, cap, nres, rows, kq, vq, shift=0.0, scale=1.0):
        self.outer, self.C, self.tq, self.cap, self.nres, self.rows = outer, C, tq, cap, nres, rows
        self.kq, self.vq = kq, vq
        self.k, self.K = self._one(rng, kq, shift, scale)
        self.v, self.V = self._one(rng, vq, shift, scale)

    def _one(self, rng, oq, shift, scale):
        o, C, tq, cap = self.outer, self.C, self.tq, self.cap
        x = W.to_bf16_bits((rng.standard_normal((o, tq, C)) * scale + shift).astype(np.float32))
        r = W.to_bf16_bits((rng.standard_normal((o, self.rows, C)) * scale + shift).astype(np.float32))
        r[:, self.nres:] = 0x7FC0                                    # NaN behind the filled rows
        mr, mc = meta_rows(oq, cap, C)
        mdt = {O.F32: np.float32, O.BF16: np.uint16, O.I8: np.int8}
        codes = np.full((o, cap, C * oq.bits // 8), 0xFF, np.uint8)
        sc = np.frombuffer(b"\xff" * (o * mr * mc * np.dtype(mdt[oq.scale_dtype]).itemsize),
                           mdt[oq.scale_dtype]).reshape(o, mr, mc).copy()
        ze = None
        if oq.zero_dtype != O.NONE:
            ze = np.frombuffer(b"\xff" * (o * mr * mc * np.dtype(mdt[oq.zero_dtype]).itemsize),
                               mdt[oq.zero_dtype]).reshape(o, mr, mc).copy()
        rows = np.zeros((o, 0, C))
        if tq:
            qt = O.quantize(x, O.BF16, oq)
            n = meta_rows(oq, tq, C)[0]
            codes[:, :tq] = qt.codes.reshape(o, tq, -1)
            sc[:, :n] = qt.scale.reshape(o, n, mc)
            if ze is not None:
                ze[:, :n] = qt.zero.reshape(o, n, mc)
            rows = bf16_to_f64(O.dequantize(qt, x.shape, oq, O.BF16))
        return [codes, sc, ze, r], np.concatenate([rows, bf16_to_f64(r[:, :self.nres])], 1)

    @property
    def T(self):
        return self.tq + self.nres

    def device(self, b, kv_heads=1, first=None):
        """(KVCache, the uint8 device tensors behind it)"""
        import torch

        def up(a):
            return None if a is None else torch.from_numpy(np.ascontiguousarray(a).view(np.uint8).ravel().copy()).cuda()
        return b.KVCache(k=tuple(up(a) for a in self.k), v=tuple(up(a) for a in self.v),
                         shape=(self.outer, self.cap, self.C), kqp=kq_of(b, self.kq), vqp=kq_of(b, self.vq),
                         tq=self.tq, nres=self.nres, resid_rows=self.rows, kv_heads=kv_heads,
                         first=None if first is None else torch.from_numpy(np.asarray(first, np.int32)).cuda())


def logits(q, K, first, kv_heads):
    """(x, mag): logits [outer, n, group, T] in binary64 (-inf: not seen) and
    sum_c |q_c k_c| / sqrt(C); q [batch, n, kv_heads * group, C] binary64."""
    B, n, H, C = q.shape
    outer, T, _ = K.shape
    G = H // kv_heads
    qs = q.reshape(B, n, kv_heads, G, C).transpose(0, 2, 1, 3, 4).reshape(outer, n, G, C)
    x = np.einsum("oijc,otc->oijt", qs, K) / np.sqrt(C)
    mag = np.einsum("oijc,otc->oijt", np.abs(qs), np.abs(K)) / np.sqrt(C)
    t = np.arange(T)
    f = np.zeros(outer, np.int64) if first is None else np.maximum(np.asarray(first, np.int64), 0)
    seen = (t >= f[:, None, None, None]) & (t <= T - n + np.arange(n)[:, None, None])
    return np.where(seen, x, -np.inf), np.where(seen, mag, 0.0)


def to_rows(x, kv_heads):
    """[outer, n, group, ...] -> [batch, n, kv_heads * group, ...]"""
    o, n, G = x.shape[:3]
    y = x.reshape(o // kv_heads, kv_heads, n, G, *x.shape[3:])
    return np.moveaxis(y, 1, 2).reshape(o // kv_heads, n, kv_heads * G, *x.shape[3:])


def softmax(x):
    """(p, lse) over the last axis; rows that see nothing: zeros and -inf."""
    m = x.max(-1, keepdims=True) if x.shape[-1] else np.full(x.shape[:-1] + (1,), -np.inf)
    e = np.exp(x - np.where(np.isinf(m), 0.0, m))
    s = e.sum(-1, keepdims=True)
    with np.errstate(divide="ignore"):
        lse = (np.where(np.isinf(m), 0.0, m) + np.log(s))[..., 0]
    return e / np.where(s > 0, s, 1.0), lse


# A score product adds C exact bf16 x bf16 products in float32; the tensor
# cores may truncate, so a step counts 2^-23.  Scaling to base 2, subtracting
# the maximum and the 2-ulp 2^x add a few more of the logit's size.
def logit_error(mag, x, C):
    """Bound on |computed - true| natural-log logits of a row, over its tokens."""
    big = np.where(np.isinf(x), 0.0, np.abs(x)).max(-1, initial=0.0)
    return (C + 8) * 2.0 ** -23 * mag.max(-1, initial=0.0) + 8 * 2.0 ** -23 * (big + 1.0)
