"""Serving many requests over the quantized cache, as cases to be measured.

Three operators that a serving loop needs beside the streaming cache's:

 prompts  causal attention over a batch of prompts, packed one behind the other
          without padding, from bf16 keys and values: what runs before there is
          a cache.  Outputs and log-sum-exps;
 fill     those prompts' keys and values into a new streaming cache: quantized
          store, bf16 buffer, and the left padding that aligns their ends;
 shared   attention of a batch over a quantized prefix that all its requests
          share, joined with the attention to tokens of each request's own: a
          streaming cache, or the (out, lse) that `prompts` gave.

With `own` false, run() computes them in elementary torch operations, in
float32 (fill: the format's own arithmetic, which is float32); with `own` true it
calls the library.
"""
import math
import random

import torch

own = False

# Layout of a case.  op: the operator; kv_heads heads of keys and values, `group`
# query heads each, `C` channels.  The lengths of the `batch` prompts (fill,
# prompts) or of what each request has of its own (shared) are spread over their
# logarithm between `shortest` and `longest`; `lens` numbers the draw.  fused:
# q, k and v are views of one projection's output.  Stores: `bits`, `sym`: the
# code format; g: the key group and the block that leaves the buffer, gv: the
# value group; the newest 128 tokens stay in bf16.  fill: `tokens` is the cache's
# length.  shared: `prefix` tokens; n queries a request; `joined`: own tokens come
# as (out, lse).
_FORMAT = {"bits": 4, "sym": False, "g": 64, "gv": 64}
_HEADS = {"kv_heads": 8, "group": 4, "C": 128}
_RESIDUAL = 128


def _case(name, **kw):
    c = {**({"name": name} if name else {}), "lens": 1, **_HEADS, **kw}
    return c if c["op"] == "prompts" else {**c, **{k: v for k, v in _FORMAT.items() if k not in c}}


def listed():
    return [
        # a single question: launch latency
        _case("prompt of 17 tokens", op="prompts", batch=1, shortest=17, longest=17, fused=True),
        # a batch of chat turns as one prefill, out of a fused projection
        _case("64 ragged prompts", op="prompts", batch=64, shortest=16, longest=2000, fused=True),
        # small heads, one query head each, odd lengths
        _case("5 prompts, small heads", op="prompts", batch=5, shortest=1501, longest=4001, kv_heads=12, group=1, C=64,
              fused=False),
        # one long document
        _case("prompt of 32768 tokens", op="prompts", batch=1, shortest=32768, longest=32768, fused=False),
        # a single question enters an empty cache: launch latency
        _case("fill, 100 tokens", op="fill", batch=1, shortest=100, longest=100, tokens=100, fused=True),
        # the chat turns
        _case("fill, 64 ragged prompts", op="fill", batch=64, shortest=16, longest=2000, tokens=2000, fused=True),
        # long documents, two-bit symmetric codes
        _case("fill, 4 long prompts, 2 bits", op="fill", batch=4, shortest=9000, longest=32768, tokens=32768, bits=2, sym=True,
              g=32, gv=32, fused=False),
        # one token each of a few requests behind a short system prompt: launch latency
        _case("shared, 4 requests, short", op="shared", batch=4, n=1, prefix=1000, shortest=20, longest=90, joined=False),
        # a decode step of a chat batch
        _case("shared, 64 requests", op="shared", batch=64, n=1, group=8, prefix=8192, shortest=50, longest=1500, joined=False),
        # drafts to be verified, two-bit symmetric codes
        _case("shared, 16 requests, 5 drafts", op="shared", batch=16, n=5, prefix=16500, shortest=100, longest=700,
              joined=False, bits=2, sym=True),
        # many short questions about one long document
        _case("shared, 128 requests, long", op="shared", batch=128, n=1, prefix=131072, shortest=30, longest=400, joined=False),
        # the prompts of a batch behind its prefix: their own tokens are attended to before
        _case("shared, prompts joined", op="shared", batch=1, n=4001, prefix=16384, shortest=4001, longest=4001, joined=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prompts", "fill", "shared"])
    c = {"op": op, "lens": rng.randrange(1 << 20), "kv_heads": rng.choice([1, 2, 4, 8, 8]),
         "group": rng.choice([1, 2, 3, 4, 5, 7, 8, 8, 16]), "C": rng.choice([64, 128, 128])}
    if op != "prompts":
        c.update(bits=rng.choice([4, 4, 2]), sym=rng.random() < 0.25, g=rng.choice([32, 64, 64, 128]),
                 gv=rng.choice([v for v in (32, 64, 128) if v <= c["C"]]))
    c["batch"] = _log_int(rng, 1, 128)
    if op == "shared":
        c["joined"] = rng.random() < 0.25
        c["prefix"] = _log_int(rng, 1, 131072)
        c["longest"] = _log_int(rng, 1, 65536 // c["batch"])
        c["shortest"] = rng.randrange(1, c["longest"] + 1)
        rows = c["batch"] * c["kv_heads"] * c["group"]
        most = max(1, min(4096, (1 << 31) // (rows * (c["prefix"] + c["longest"]))))
        c["n"] = 1 if rng.random() < 0.5 else _log_int(rng, 1, most)
        return c
    most = min(32768, 65536 // c["batch"])
    if op == "prompts":                                     # no more products than the longest listed prompt's
        most = min(most, int((2.0 ** 42 / (c["batch"] * c["kv_heads"] * c["group"] * c["C"])) ** 0.5))
    c["longest"] = _log_int(rng, 1, most)
    c["shortest"] = rng.randrange(1, c["longest"] + 1)
    c["fused"] = rng.random() < 0.5
    if op == "fill":
        c["tokens"] = max(1, c["longest"] - rng.choice([0, 0, 0, c["longest"] // 3]) + rng.choice([0, 0, 50]))
    return c


def _lens(case):
    """The lengths of the case's prompts, or of its requests' own tokens."""
    lo, hi, rng = case["shortest"], case["longest"], random.Random(case["lens"])
    lens = [_log_int(rng, lo, hi) for _ in range(case["batch"])]
    lens[rng.randrange(len(lens))] = hi
    return lens


def _split(case, T):
    """(store tokens, buffer tokens) of a cache of T tokens, and the rows of its buffer."""
    g = case["g"]
    tq = g * max(0, (T - _RESIDUAL) // g)
    return tq, T - tq, _RESIDUAL + g


# ---- inputs ------------------------------------------------------------------

def _divide(x, n):
    return x / torch.full((), float(n), device=x.device)       # a tensor: a division by a number may be by its reciprocal


def _constants(lo, hi, case):
    """Scale and zero point, float32 holding what bf16 stores, of groups of extremes lo and hi."""
    floor = torch.full((), 1e-8, device=lo.device)
    if case["sym"]:
        top = (1 << (case["bits"] - 1)) - 1
        return _divide(torch.maximum(torch.maximum(-lo, hi), floor), top).bfloat16().float(), None
    s = _divide(torch.maximum(hi - lo, floor), (1 << case["bits"]) - 1).bfloat16().float()
    return s, (-(lo / s)).round().bfloat16().float()


def _codes(x, s, z, case):
    if case["sym"]:
        top = (1 << (case["bits"] - 1)) - 1
        return (x / s).round().clamp(-top, top).int()
    return ((x / s).round() + z).clamp(0, (1 << case["bits"]) - 1).int()


def _pack(codes, bits):
    per = 8 // bits
    c = (codes & ((1 << bits) - 1)).reshape(*codes.shape[:-1], codes.shape[-1] // per, per)
    return sum(c[..., k] << (bits * k) for k in range(per)).to(torch.uint8)


def _empty_cache(case, O, T, gen):
    """Buffers of a cache for T tokens a slice; what no token fills holds other tokens' bytes."""
    C, dev = case["C"], "cuda"
    tq, _, rows = _split(case, T)
    cap = max(tq, case["g"])
    s = {}
    for w, shape in (("k", (O, cap // case["g"], C)), ("v", (O, cap, C // case["gv"]))):
        s[w + "_codes"] = torch.randint(0, 256, (O, cap, C * case["bits"] // 8), generator=gen, device=dev, dtype=torch.uint8)
        s[w + "_scale"] = torch.ones(shape, device=dev, dtype=torch.bfloat16)
        s[w + "_zero"] = None if case["sym"] else torch.zeros(shape, device=dev, dtype=torch.bfloat16)
        s[w + "_resid"] = torch.randn((O, rows, C), generator=gen, device=dev).bfloat16()
    return s


def _loud(x, gen):
    """A few loud channels, as keys have."""
    x[..., torch.randint(0, x.shape[-1], (4,), generator=gen, device=x.device)] *= 4.0
    return x


def _full_cache(case, O, T, first, gen):
    """A cache of T tokens a slice, the ones before first[o] padding."""
    C, g, gv = case["C"], case["g"], case["gv"]
    tq, nres, rows = _split(case, T)
    s = _empty_cache(case, O, T, gen)
    k = _loud(torch.randn((O, tq + rows, C), generator=gen, device="cuda"), gen).bfloat16()
    v = torch.randn((O, tq + rows, C), generator=gen, device="cuda").bfloat16()
    s["k_resid"], s["v_resid"] = k[:, tq:].contiguous(), v[:, tq:].contiguous()
    s["first"] = torch.tensor(first, dtype=torch.int32, device="cuda")
    if tq:
        for w, x, axis in (("k", k[:, :tq].float().reshape(O, tq // g, g, C), 2),
                           ("v", v[:, :tq].float().reshape(O, tq, C // gv, gv), 3)):
            scale, zero = _constants(x.amin(axis, keepdim=True), x.amax(axis, keepdim=True), case)
            s[w + "_codes"][:, :tq] = _pack(_codes(x, scale, zero, case).reshape(O, tq, C), case["bits"])
            n = scale.squeeze(axis).shape[1]
            s[w + "_scale"][:, :n] = scale.squeeze(axis).bfloat16()
            if zero is not None:
                s[w + "_zero"][:, :n] = zero.squeeze(axis).bfloat16()
    return {**s, "tq": tq, "nres": nres, "rows": rows}


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    Hk, G, C, lens, op = case["kv_heads"], case["group"], case["C"], _lens(case), case["op"]
    st = {"case": case, "lens": lens}
    if op == "shared":
        B, n, H = case["batch"], case["n"], Hk * G
        st["q"] = (1.5 * torch.randn((B, n, H, C), generator=gen, device="cuda")).bfloat16()
        st["prefix"] = _full_cache(case, Hk, case["prefix"], [0] * Hk, gen)
        if case["joined"]:
            st["out"] = (0.2 * torch.randn((B, n, H, C), generator=gen, device="cuda")).bfloat16()
            st["lse"] = math.log(max(lens)) + torch.randn((B, n, H), generator=gen, device="cuda")
        else:
            st["cache"] = _full_cache(case, B * Hk, max(lens), [max(lens) - x for x in lens for _ in range(Hk)], gen)
        return st
    total, heads = sum(lens), (G * Hk if op == "prompts" else 0)
    x = torch.randn((total, heads + 2 * Hk, C), generator=gen, device="cuda")
    _loud(x[:, heads:heads + Hk], gen)
    x[:, :heads] *= 1.5
    x = x.bfloat16()
    st["q"], st["k"], st["v"] = (t if case["fused"] else t.contiguous() for t in x.split([heads, Hk, Hk], 1))
    st["starts"] = torch.tensor([0] + lens, device="cuda").cumsum(0).int()
    if op == "fill":
        st["cache"] = _empty_cache(case, case["batch"] * Hk, case["tokens"], gen)
        st["cache"]["first"] = torch.zeros(case["batch"] * Hk, dtype=torch.int32, device="cuda")
    return st


# ---- the plain forms ---------------------------------------------------------

def _softmax_product(x, v):
    """(out, lse) of logits x [..., rows, tokens], changed in place, over values v."""
    top = x.amax(-1, keepdim=True)
    x = x.sub_(top.clamp_min(-3e38)).exp_()
    total = x.sum(-1, keepdim=True)
    return (x @ v) / total.clamp_min(1e-38), (top + total.log()).squeeze(-1)


_MOST = 1 << 30                                            # scores held at once


def _prompts(s):
    """Prompts of like lengths together, padded to the longest of them; long ones in pieces of their queries."""
    c, lens = s["case"], s["lens"]
    Hk, G, C = c["kv_heads"], c["group"], c["C"]
    out = torch.empty((sum(lens), Hk * G, C), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((sum(lens), Hk * G), device="cuda")
    for size in sorted({x.bit_length() for x in lens}):
        ids = torch.tensor([i for i, x in enumerate(lens) if x.bit_length() == size], device="cuda")
        n = max(x for x in lens if x.bit_length() == size)
        at = s["starts"].long()[ids][:, None] + torch.arange(n, device="cuda")
        live = at < s["starts"].long()[ids + 1][:, None]
        rows = at.clamp_max(sum(lens) - 1)
        k, v = (s[w][rows].float().transpose(1, 2).unsqueeze(2) for w in "kv")         # [ids, Hk, 1, n, C]
        step = max(1, min(n, _MOST // (len(ids) * Hk * G * n)))
        for i in range(0, n, step):
            q = s["q"][rows[:, i:i + step]].float().reshape(len(ids), -1, Hk, G, C).permute(0, 2, 3, 1, 4)
            end = i + q.shape[3]
            x = (q @ k[..., :end, :].transpose(3, 4)).mul_(C ** -0.5)
            t = torch.arange(end, device="cuda")
            y, z = _softmax_product(x.masked_fill_(t > t[i:, None], -math.inf), v[..., :end, :])
            some = live[:, i:end]
            out[at[:, i:end][some]] = y.permute(0, 3, 1, 2, 4).flatten(2, 3)[some].bfloat16()
            lse[at[:, i:end][some]] = z.permute(0, 3, 1, 2).flatten(2, 3)[some]
    return out, lse


def _fill(s):
    c, T, cache = s["case"], s["case"]["tokens"], s["cache"]
    Hk, C, g, gv, B = c["kv_heads"], c["C"], c["g"], c["gv"], c["batch"]
    tq, nres, _ = _split(c, T)
    starts = s["starts"].long()
    first = (T - (starts[1:] - starts[:-1])).clamp_min(0)
    cache["first"].copy_(first.repeat_interleave(Hk))
    t = torch.arange(T, device="cuda")
    at = (starts[1:, None] - T + t).clamp_min(0)
    live = (t >= first[:, None]).repeat_interleave(Hk, 0)                               # [B Hk, T]
    for w in "kv":
        x = s[w][at].transpose(1, 2).reshape(B * Hk, T, C)
        buf = cache[w + "_resid"][:, :nres]
        buf.copy_(torch.where(live[:, tq:, None], x[:, tq:], buf))
        if tq == 0:
            continue
        x, seen = x[:, :tq].float(), live[:, :tq, None].expand(-1, -1, C)
        shape, axis = ((B * Hk, tq // g, g, C), 2) if w == "k" else ((B * Hk, tq, C // gv, gv), 3)
        x, seen = x.reshape(shape), seen.reshape(shape)
        lo = x.masked_fill(~seen, math.inf).amin(axis, keepdim=True)
        hi = x.masked_fill(~seen, -math.inf).amax(axis, keepdim=True)
        some = seen.any(axis)
        scale, zero = _constants(lo, hi, c)
        codes = _pack(_codes(x, scale, zero, c).reshape(B * Hk, tq, C), c["bits"])
        to = cache[w + "_codes"][:, :tq]
        to.copy_(torch.where(live[:, :tq, None], codes, to))
        for name, m in (("_scale", scale), ("_zero", zero)):
            if m is not None:
                to = cache[w + name][:, :some.shape[1]]
                to.copy_(torch.where(some, m.squeeze(axis).bfloat16(), to))
    return _buffers(cache)


def _buffers(cache):
    names = [w + n for w in "kv" for n in ("_codes", "_scale", "_zero", "_resid")]
    return [cache["first"]] + [cache[n] for n in names if cache[n] is not None]


def _dequant(cache, c, w):
    """[slices, tokens, C] float32: the bf16 rows that the cache stands for."""
    bits, tq = c["bits"], cache["tq"]
    codes = cache[w + "_codes"][:, :tq]
    shift = torch.arange(0, 8, bits, device=codes.device, dtype=torch.int32)
    x = ((codes.int()[..., None] >> shift) & ((1 << bits) - 1)).flatten(-2)
    if c["sym"]:
        x = torch.where(x >= 1 << (bits - 1), x - (1 << bits), x)
    x = x.float()
    ax, rep = (1, c["g"]) if w == "k" else (2, c["gv"])
    used = slice(0, tq // c["g"] if w == "k" else tq)
    if not c["sym"]:
        x = x - cache[w + "_zero"][:, used].float().repeat_interleave(rep, ax)
    x = x * cache[w + "_scale"][:, used].float().repeat_interleave(rep, ax)
    return torch.cat([x.bfloat16(), cache[w + "_resid"][:, :cache["nres"]]], 1).float()


def _shared(s):
    c = s["case"]
    B, n, Hk, G, C = c["batch"], c["n"], c["kv_heads"], c["group"], c["C"]
    q = s["q"].float().reshape(B, n, Hk, G, C)

    def prefix(rows):                                                                   # [Hk, rows, C]
        x = (rows @ k.transpose(1, 2)).mul_(C ** -0.5)
        return _softmax_product(x, v)

    k, v = (_dequant(s["prefix"], c, w) for w in "kv")
    rows = q.permute(2, 0, 1, 3, 4).reshape(Hk, -1, C)
    step = max(1, _MOST // (Hk * k.shape[1]))
    parts = [prefix(rows[:, i:i + step]) for i in range(0, rows.shape[1], step)]
    y0 = torch.cat([p[0] for p in parts], 1).reshape(Hk, B, n, G, C).permute(1, 2, 0, 3, 4).reshape(B, n, Hk * G, C)
    z0 = torch.cat([p[1] for p in parts], 1).reshape(Hk, B, n, G).permute(1, 2, 0, 3).reshape(B, n, Hk * G)
    if c["joined"]:
        y1, z1 = s["out"].float(), s["lse"]
    else:
        k, v = (_dequant(s["cache"], c, w).reshape(B, Hk, -1, C) for w in "kv")
        T = k.shape[2]
        x = (q.permute(0, 2, 1, 3, 4).reshape(B, Hk, n * G, C) @ k.transpose(2, 3)).mul_(C ** -0.5)
        t = torch.arange(T, device="cuda")
        last = (T - n + torch.arange(n, device="cuda")).repeat_interleave(G)
        hidden = (t < s["cache"]["first"].reshape(B, Hk, 1, 1)) | (t > last[:, None])
        y1, z1 = _softmax_product(x.masked_fill_(hidden, -math.inf), v)
        y1 = y1.reshape(B, Hk, n, G, C).transpose(1, 2).reshape(B, n, Hk * G, C)
        z1 = z1.reshape(B, Hk, n, G).transpose(1, 2).reshape(B, n, Hk * G)
    lse = torch.logaddexp(z0, z1)
    out = y0 * (z0 - lse).exp()[..., None] + y1 * (z1 - lse).exp()[..., None]
    return out.bfloat16(), lse


# ---- the library -------------------------------------------------------------

def _own_cache(b, s, c, bufs, tq, nres, rows):
    kw = dict(scale_dtype=b.BF16, residual=_RESIDUAL)
    if c["sym"]:
        kq = b.QParams.sym(c["bits"], axis=b.ALONG_T, group=c["g"], **kw)
        vq = b.QParams.sym(c["bits"], axis=b.ALONG_C, group=c["gv"], **kw)
    else:
        kq = b.QParams.asym(c["bits"], 0, (1 << c["bits"]) - 1, axis=b.ALONG_T, group=c["g"], zero_dtype=b.BF16, **kw)
        vq = b.QParams.asym(c["bits"], 0, (1 << c["bits"]) - 1, axis=b.ALONG_C, group=c["gv"], zero_dtype=b.BF16, **kw)
    return b.KVCache(*[tuple(bufs[w + n] for n in ("_codes", "_scale", "_zero", "_resid")) for w in "kv"],
                     shape=(bufs["k_codes"].shape[0], bufs["k_codes"].shape[1], c["C"]), kqp=kq, vqp=vq, tq=tq, nres=nres,
                     resid_rows=rows, kv_heads=c["kv_heads"], first=bufs["first"])


def _own(s):
    from kv_cache_quantization_kvq_gb300 import binding as b
    c = s["case"]
    if c["op"] == "prompts":
        return b.attend_prompts(s["q"], s["k"], s["v"], s["starts"])
    if c["op"] == "fill":
        cache = _own_cache(b, s, c, s["cache"], 0, 0, _split(c, c["tokens"])[2])
        b.fill_prompts(s["k"], s["v"], s["starts"], cache, c["tokens"])
        return _buffers(s["cache"])
    caches = [_own_cache(b, s, c, x, x["tq"], x["nres"], x["rows"]) for x in (s["prefix"], s.get("cache")) if x]
    if c["joined"]:
        return b.attend_shared(s["q"], caches[0], own=(s["out"], s["lse"]))
    return b.attend_shared(s["q"], *caches)


def run(state):
    if own:
        return _own(state)
    return {"prompts": _prompts, "fill": _fill, "shared": _shared}[state["case"]["op"]](state)


# ---- what a pass cannot do without --------------------------------------------

def _stored(case, T, tokens, slices_of_each):
    """Bytes of the last `tokens` tokens of a cache of length T, in a slice, times slices."""
    tq = _split(case, T)[0]
    first, C, meta = T - tokens, case["C"], 2 if case["sym"] else 4
    store = max(0, tq - first)
    groups = max(0, tq // case["g"] - first // case["g"])
    return slices_of_each * (store * (C * case["bits"] // 4 + C // case["gv"] * meta) + groups * C * meta +
                             (tokens - store) * 4 * C)


def work(case):
    Hk, G, C, lens = case["kv_heads"], case["group"], case["C"], _lens(case)
    if case["op"] == "prompts":
        rows = sum(lens) * Hk * G
        return {"bytes": rows * (4 * C + 4) + sum(lens) * Hk * 4 * C + 4 * len(lens) + 4,
                "flops": 4 * C * Hk * G * sum(x * (x + 1) // 2 for x in lens)}
    if case["op"] == "fill":
        T = case["tokens"]
        kept = [min(x, T) for x in lens]
        return {"bytes": sum(kept) * Hk * 4 * C + sum(_stored(case, T, x, Hk) for x in kept) + 4 * len(lens) * (Hk + 1) + 4,
                "flops": 0}
    n = case["n"]
    rows = case["batch"] * n * Hk * G
    b = rows * (4 * C + 4) + _stored(case, case["prefix"], case["prefix"], Hk)
    pairs = rows * case["prefix"]
    if case["joined"]:
        b += rows * (2 * C + 4)
    else:
        T = max(lens)
        b += sum(_stored(case, T, x, Hk) for x in lens) + 4 * case["batch"] * Hk
        # query i of a request of x tokens sees x - n + 1 + i of them
        pairs += Hk * G * sum((max(0, x - n + 1) + x) * (x - max(0, x - n + 1) + 1) // 2 for x in lens)
    return {"bytes": b, "flops": 4 * C * pairs}


# ---- the definitions in 64 bits ------------------------------------------------

def exact(case, seed):
    if case["op"] != "fill" and work(case)["flops"] > 4e12:
        return None
    s = prepare(case, seed)
    return {"prompts": _exact_prompts, "fill": _exact_fill, "shared": _exact_shared}[case["op"]](s)


def _exact_attention(q, k, v, seen):
    """(out, lse) of queries [rows, C] over keys and values [tokens, C]; seen(row numbers) -> [rows, tokens]."""
    out, lse = [], []
    for i in range(0, q.shape[0], 2048):
        x = q[i:i + 2048] @ k.T / math.sqrt(q.shape[1])
        x = torch.where(seen(torch.arange(i, i + x.shape[0], device=x.device)), x, -math.inf)
        z = torch.logsumexp(x, 1)
        out.append(torch.exp(x - torch.where(z.isinf(), 0.0, z)[:, None]) @ v)
        lse.append(z)
    return torch.cat(out), torch.cat(lse)


def _exact_prompts(s):
    c = s["case"]
    total, H = s["q"].shape[0], c["kv_heads"] * c["group"]
    out = torch.empty((total, H, c["C"]), dtype=torch.float64, device="cuda")
    lse = torch.empty((total, H), dtype=torch.float64, device="cuda")
    a = 0
    for n in s["lens"]:
        for head in range(H):
            kv = head // c["group"]
            out[a:a + n, head], lse[a:a + n, head] = _exact_attention(
                s["q"][a:a + n, head].double(), s["k"][a:a + n, kv].double(), s["v"][a:a + n, kv].double(),
                lambda i: torch.arange(n, device="cuda") <= i[:, None])
        a += n
    return out, lse


def _exact_fill(s):
    """Scales, zero points and buffer rows; the codes are whole numbers."""
    c, cache, T = s["case"], s["cache"], s["case"]["tokens"]
    Hk, g, gv, bits = c["kv_heads"], c["g"], c["gv"], c["bits"]
    tq, nres, _ = _split(c, T)
    new = {k: None if x is None or k.endswith("_codes") else x if k == "first" else x.double() for k, x in cache.items()}
    a = 0

    def constants(x):                                       # [..., members] -> the group's two
        if c["sym"]:
            return (x.abs().amax(-1) / (2 ** (bits - 1) - 1)).bfloat16().double(), None
        lo = x.amin(-1)
        scale = ((x.amax(-1) - lo).clamp_min(1e-8) / (2 ** bits - 1)).bfloat16().double()
        return scale, torch.round(-lo / scale).bfloat16().double()

    for b, n in enumerate(s["lens"]):
        m = min(n, T)
        for w in "kv":
            x = s[w][a + n - m:a + n].double().transpose(0, 1)                          # [Hk, m, C]
            first, o = T - m, slice(b * Hk, (b + 1) * Hk)
            new["first"][o] = first
            kept = min(nres, m)
            new[w + "_resid"][o, nres - kept:nres] = x[:, m - kept:]
            if m - kept == 0:
                continue
            x = x[:, :m - kept]                                                         # store tokens first .. tq
            if w == "v":
                scale, zero = constants(x.reshape(Hk, m - kept, -1, gv))
                where = slice(first, tq)
            else:
                head = -first % g
                parts = ([x[:, :head].transpose(1, 2)] if head else [])
                got = [constants(p) for p in parts]
                if head < x.shape[1]:
                    full = constants(x[:, head:].reshape(Hk, -1, g, c["C"]).transpose(2, 3))
                    got = [(p[:, None], z if z is None else z[:, None]) for p, z in got] + [full]
                else:
                    got = [(p[:, None], z if z is None else z[:, None]) for p, z in got]
                scale = torch.cat([p for p, _ in got], 1)
                zero = None if c["sym"] else torch.cat([z for _, z in got], 1)
                where = slice(first // g, tq // g)
            new[w + "_scale"][o, where] = scale
            if zero is not None:
                new[w + "_zero"][o, where] = zero
        a += n
    names = [w + n for w in "kv" for n in ("_codes", "_scale", "_zero", "_resid")]
    return [new["first"]] + [new[n] for n in names if cache[n] is not None]


def _value(cache, c, o, w):
    """Slice o's rows in binary64, code by code: s (code - zp) rounded to bf16, then the buffer's rows."""
    per, tq = 8 // c["bits"], cache["tq"]
    byte = cache[w + "_codes"][o, :tq].long()
    x = torch.empty((tq, c["C"]), dtype=torch.float64, device=byte.device)
    for k in range(per):
        f = torch.div(byte, 2 ** (c["bits"] * k), rounding_mode="floor") % 2 ** c["bits"]
        if c["sym"]:
            f = (f + 2 ** (c["bits"] - 1)) % 2 ** c["bits"] - 2 ** (c["bits"] - 1)
        x[:, k::per] = f.double()
    for name, sign in (("_zero", 0), ("_scale", 1)):
        m = cache[w + name]
        if m is None:
            continue
        m = m[o].double()
        if w == "k":
            m = m[torch.arange(tq, device=m.device) // c["g"]]
        else:
            m = m[:tq][:, torch.arange(c["C"], device=m.device) // c["gv"]]
        x = x * m if sign else x - m
    return torch.cat([x.bfloat16().double(), cache[w + "_resid"][o, :cache["nres"]].double()])


def _exact_shared(s):
    c = s["case"]
    B, n, Hk, G, C = c["batch"], c["n"], c["kv_heads"], c["group"], c["C"]
    out = torch.empty((B, n, Hk * G, C), dtype=torch.float64, device="cuda")
    lse = torch.empty((B, n, Hk * G), dtype=torch.float64, device="cuda")
    for h in range(Hk):
        kp, vp = _value(s["prefix"], c, h, "k"), _value(s["prefix"], c, h, "v")
        heads = slice(h * G, (h + 1) * G)
        q = s["q"][:, :, heads].reshape(-1, C).double()
        y, z = _exact_attention(q, kp, vp, lambda i: torch.ones_like(i, dtype=torch.bool)[:, None])
        y, z = y.reshape(B, n, G, C), z.reshape(B, n, G)
        for b in range(B):
            if c["joined"]:
                y1, z1 = s["out"][b, :, heads].double(), s["lse"][b, :, heads].double()
            else:
                o = b * Hk + h
                k, v = _value(s["cache"], c, o, "k"), _value(s["cache"], c, o, "v")
                t, first = torch.arange(k.shape[0], device="cuda"), max(s["lens"]) - s["lens"][b]
                y1, z1 = _exact_attention(s["q"][b, :, heads].reshape(-1, C).double(), k, v,
                                          lambda i: (t >= first) & (t <= (k.shape[0] - n + i // G)[:, None]))
                y1, z1 = y1.reshape(n, G, C), z1.reshape(n, G)
            both = torch.logaddexp(z[b], z1)
            out[b, :, heads] = y[b] * torch.exp(z[b] - both)[..., None] + y1 * torch.exp(z1 - both)[..., None]
            lse[b, :, heads] = both
    return out, lse
