"""Packed prompts for the tests of kvq_attend_prompts and kvq_fill_prompts, and
the formulas in binary64."""
import numpy as np

import stream_util as S
from kv_cache_quantization_kvq_gb300 import workloads as W


def upload_bf16(bits):
    import torch
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16).copy()).view(torch.bfloat16).cuda()


def starts_of(lens, before=0):
    return (before + np.concatenate([[0], np.cumsum(lens)])).astype(np.int32)


def packed(rng, total, heads, C, loud=0, scale=1.0):
    """bf16 bits [total, heads, C]; the first `loud` channels four times as large."""
    x = rng.standard_normal((total, heads, C)) * scale
    x[..., :loud] *= 4.0
    return W.to_bf16_bits(x.astype(np.float32))


def prompt_reference(q, k, v, group):
    """One prompt's rows in binary64, [L, heads, C] of q and [L, kv_heads, C] of k, v:
    (lse, out, sum p |v|, row's logit error) with the causal mask."""
    L, H, C = q.shape
    kk, vv = (np.repeat(x, group, 1) for x in (k, v))
    x = np.einsum("ihc,jhc->hij", q, kk) / np.sqrt(C)
    mag = np.einsum("ihc,jhc->hij", np.abs(q), np.abs(kk)) / np.sqrt(C)
    seen = np.arange(L) <= np.arange(L)[:, None]
    x, mag = np.where(seen, x, -np.inf), np.where(seen, mag, 0.0)
    p, lse = S.softmax(x)
    out, absout = (np.einsum("hij,jhc->ihc", p, y) for y in (vv, np.abs(vv)))
    return lse.T, out, absout, 2.0 * S.logit_error(mag, x, C).T


U = 2.0 ** -8                                    # the largest relative error of a rounding to bf16


def tolerances(lse, out, absout, e, T):
    """Of lse and out: as test_stream_attend_gpu.py derives them."""
    sums = (T + 64) * 2.0 ** -23
    finite = np.where(np.isfinite(lse), np.abs(lse), 0.0)
    return e + sums + 4 * 2.0 ** -23 * (finite + 1.0), (U + e + sums)[..., None] * absout + U * np.abs(out)


def close(got, want, tol, what):
    with np.errstate(invalid="ignore"):
        bad = ~(np.abs(got - want) <= tol)
    bad &= ~((got == want) | (np.isnan(got) & np.isnan(want)))
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, first at {np.argwhere(bad)[0]}: " \
                          f"{got[bad][0]} for {want[bad][0]} (tolerance {np.broadcast_to(tol, bad.shape)[bad][0]})"


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)
