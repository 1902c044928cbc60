"""The streaming quantized cache's operators, as cases to be measured.

Three operators that a serving loop runs on one layer's quantized KV cache
(the store and the bf16 buffer that kvq_append_kv fills):

 attend   attention of the n newest tokens' queries over the cache, causal,
          with a left padding per slice: the outputs and the log-sum-exp of
          every query row;
 weights  the attention weight that those queries give every token, added to
          the running score of the token;
 evict    the blocks with the least accumulated score leave the cache, the
          others close ranks (out of place here, so that a pass can be
          repeated on the same state).

With `own` false, run() computes them in elementary torch operations, in
float32 on the rows that the format stands for; with `own` true it calls the
library.
"""
import math

import torch

own = False

# Layout of a case.  op: the operator; batch x kv_heads KV slices, each read by
# `group` query heads of `C` channels; the store holds `tq` quantized tokens of
# `cap` and the buffer `nres` bf16 tokens of `rows`; n: queries (the newest
# tokens); pad: the left padding of the batch's last sequence (the others have
# less); bits, sym: the code format; g: the key group, gv: the value group.
_BASE = {"bits": 4, "sym": False, "g": 64, "gv": 64, "C": 128, "pad": 0}


def _case(name, **kw):
    return {**({"name": name} if name else {}), **_BASE, **kw}


def listed():
    return [
        # one token of a short chat: launch latency
        _case("attend one token, short", op="attend", batch=1, kv_heads=8, group=4, n=1, tq=960, cap=1024, nres=77,
              rows=192),
        # one decode step of 8 sequences x 8 KV heads over 8192 tokens (the KIVI workload), 8 query heads each
        _case("attend one token, 64 slices", op="attend", batch=8, kv_heads=8, group=8, n=1, tq=8064, cap=8192,
              nres=128, rows=192),
        # one token of one long conversation, padded: few rows, a long axis
        _case("attend one token, long", op="attend", batch=1, kv_heads=8, group=4, n=1, tq=131072, cap=135168,
              nres=191, rows=192, pad=1000),
        # five drafted tokens to be verified at once, two-bit cache, symmetric codes, ragged batch
        _case("attend five drafts, 2 bits", op="attend", batch=4, kv_heads=8, group=4, n=5, tq=16320, cap=16384,
              nres=133, rows=192, bits=2, sym=True, pad=4100),
        # a prompt's first chunk, short and ragged, small heads
        _case("attend prompt, ragged", op="attend", batch=4, kv_heads=8, group=2, n=1000, tq=896, cap=1024, nres=104,
              rows=192, C=64, gv=32, pad=333),
        # a chunk of a long prompt over what the cache holds already
        _case("attend chunk of a long prompt", op="attend", batch=1, kv_heads=8, group=4, n=4096, tq=32640, cap=32768,
              nres=128, rows=192),
        # the weights of one decode step of the KIVI workload
        _case("weights one token, 64 slices", op="weights", batch=8, kv_heads=8, group=8, n=1, tq=8064, cap=8192,
              nres=128, rows=192),
        # the last 63 queries of a prompt as the observation window
        _case("weights of a window", op="weights", batch=2, kv_heads=8, group=4, n=63, tq=32704, cap=32768, nres=70,
              rows=192, pad=5000),
        # every query of a prompt's chunk
        _case("weights of a chunk", op="weights", batch=1, kv_heads=8, group=4, n=2048, tq=16320, cap=16384, nres=64,
              rows=192),
        # a short cache loses one block: launch latency
        _case("evict one block, short", op="evict", batch=1, kv_heads=8, group=1, n=0, tq=1088, cap=1152, nres=100,
              rows=192, budget=16, window=2),
        # a batch over its budget
        _case("evict an eighth, 64 slices", op="evict", batch=8, kv_heads=8, group=1, n=0, tq=8192, cap=8448, nres=130,
              rows=192, budget=112, window=8),
        # a prompt of 32768 tokens cut down to its quarter
        _case("evict to a quarter, long", op="evict", batch=4, kv_heads=32, group=1, n=0, tq=32768, cap=32768, nres=37,
              rows=192, budget=128, window=4, pad=700),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "weights", "weights", "evict"])
    c = dict(_BASE, op=op, bits=rng.choice([4, 4, 4, 2]), sym=rng.random() < 0.25, C=rng.choice([64, 128, 128]))
    c["g"] = rng.choice([32, 64, 64, 128])
    c["gv"] = rng.choice([v for v in (32, 64, 128) if v <= c["C"]])
    c["batch"], c["kv_heads"] = rng.choice([1, 1, 2, 3, 4, 8]), rng.choice([1, 2, 4, 8, 8])
    slices = c["batch"] * c["kv_heads"]
    c["rows"] = 128 + c["g"]
    c["nres"] = rng.randrange(0, c["rows"])
    if op == "evict":
        blocks = max(2, _log_int(rng, 512, min(131072, 4194304 // slices)) // c["g"])
        c.update(group=1, n=0, tq=blocks * c["g"])
        c["budget"] = rng.randrange(1, blocks + 1)
        c["window"] = rng.randrange(0, min(c["budget"], 9))
    else:
        c["group"] = rng.choice([1, 2, 3, 4, 5, 7, 8, 8, 16])
        T = _log_int(rng, 256, min(131072, 2097152 // slices))
        c["tq"] = T // c["g"] * c["g"]
        T = max(1, c["tq"] + c["nres"])
        c["nres"] = T - c["tq"]
        # a third single tokens, a third short runs, a third chunks of any length
        most = max(1, min(T, 4096, (1 << 31) // (slices * c["group"] * T)))
        kind = rng.randrange(3)
        c["n"] = 1 if kind == 0 else min(most, rng.randrange(2, 17)) if kind == 1 else _log_int(rng, 1, most)
    c["cap"] = c["tq"] + c["g"] * rng.randrange(0, 4)
    if c["batch"] > 1 and rng.random() < 0.6:
        c["pad"] = rng.randrange(0, c["tq"] + c["nres"])
    return c


def _first(case):
    """The left padding of every KV slice: from 0 for the first sequence to `pad` for the last."""
    B = case["batch"]
    return [case["pad"] * b // max(1, B - 1) if B > 1 else case["pad"] for b in range(B) for _ in range(case["kv_heads"])]


def _quantize(x, bits, sym, g):
    """[outer, T, C] in groups of g along the middle axis: codes, scale and zero point in the values' types."""
    o, t, c = x.shape
    x = x.reshape(o, t // g, g, c)
    if sym:
        top = (1 << (bits - 1)) - 1
        s = (x.abs().amax(2, keepdim=True) / top).clamp_min(1e-8).bfloat16().float()
        return (x / s).round().clamp(-top, top).reshape(o, t, c).int(), s[:, :, 0].bfloat16(), None
    top = (1 << bits) - 1
    lo, hi = x.amin(2, keepdim=True), x.amax(2, keepdim=True)
    s = ((hi - lo) / top).clamp_min(1e-8).bfloat16().float()
    z = (-lo / s).round().bfloat16().float()
    return ((x / s).round() + z).clamp(0, top).reshape(o, t, c).int(), s[:, :, 0].bfloat16(), z[:, :, 0].bfloat16()


def _pack(codes, bits):
    per = 8 // bits
    c = (codes & ((1 << bits) - 1)).reshape(*codes.shape[:-1], codes.shape[-1] // per, per)
    return sum(c[..., k] << (bits * k) for k in range(per)).to(torch.uint8)


def _cache(case, gen):
    O, C, tq, cap, g, gv = (case["batch"] * case["kv_heads"], case["C"], case["tq"], case["cap"], case["g"], case["gv"])
    bits, sym, dev = case["bits"], case["sym"], "cuda"

    def randn(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    k = randn(O, tq, C)
    loud = torch.randint(0, C, (4,), generator=gen, device=dev)
    k[..., loud] *= 4.0                                     # a few loud channels, as keys have
    v = randn(O, tq, C)
    s = {"k_codes": torch.randint(0, 256, (O, cap, C * bits // 8), generator=gen, device=dev, dtype=torch.uint8),
         "v_codes": torch.randint(0, 256, (O, cap, C * bits // 8), generator=gen, device=dev, dtype=torch.uint8),
         "k_scale": torch.ones(O, -(-cap // g), C, device=dev, dtype=torch.bfloat16),
         "v_scale": torch.ones(O, cap, C // gv, device=dev, dtype=torch.bfloat16),
         "k_zero": None, "v_zero": None}
    if not sym:
        s["k_zero"], s["v_zero"] = torch.zeros_like(s["k_scale"]), torch.zeros_like(s["v_scale"])
    if tq:
        codes, scale, zero = _quantize(k, bits, sym, g)
        s["k_codes"][:, :tq], s["k_scale"][:, :tq // g] = _pack(codes, bits), scale
        if not sym:
            s["k_zero"][:, :tq // g] = zero
        codes, scale, zero = _quantize(v.reshape(O * tq, C, 1), bits, sym, gv)
        s["v_codes"][:, :tq] = _pack(codes.reshape(O, tq, C), bits)
        s["v_scale"][:, :tq] = scale.reshape(O, tq, C // gv)
        if not sym:
            s["v_zero"][:, :tq] = zero.reshape(O, tq, C // gv)
    s["k_resid"], s["v_resid"] = randn(O, case["rows"], C).bfloat16(), randn(O, case["rows"], C).bfloat16()
    s["k_resid"][..., loud] *= 4.0
    s["first"] = torch.tensor(_first(case), dtype=torch.int32, device=dev)
    return s


_STORE = ("k_codes", "k_scale", "k_zero", "v_codes", "v_scale", "v_zero")


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    O, C, T = case["batch"] * case["kv_heads"], case["C"], case["tq"] + case["nres"]
    st = {"case": case, **_cache(case, gen)}
    if case["op"] == "evict":
        # accumulated weights: a few heavy hitters, nothing on the padding
        sc = torch.exp(2.5 * torch.randn((O, case["cap"] + case["rows"]), generator=gen, device="cuda"))
        at = torch.arange(sc.shape[1], device="cuda")[None]
        sc[(at < st["first"][:, None]) | (at >= T)] = 0.0
        st["scores"], st["scores_out"] = sc, torch.zeros_like(sc)
        st["dst"] = {k: None if st[k] is None else torch.zeros_like(st[k]) for k in _STORE}
        st["keep"] = torch.empty((O, min(case["budget"], case["tq"] // case["g"])), dtype=torch.int32, device="cuda")
        st["first_out"] = torch.empty_like(st["first"])
        return st
    q = torch.randn((case["batch"], case["n"], case["kv_heads"] * case["group"], C), generator=gen, device="cuda")
    st["q"] = (1.5 * q).bfloat16()
    if case["op"] == "weights":
        st["scores"] = torch.rand((O, case["cap"] + case["rows"]), generator=gen, device="cuda")
        st["lse"] = _attend(st)[1]
    return st


# ---- the plain forms ---------------------------------------------------------

def _dequant(s, which, along_t):
    """[outer, tq + nres, C] float32: the bf16 rows that the cache stands for."""
    c = s["case"]
    bits, tq = c["bits"], c["tq"]
    codes = s[which + "_codes"][:, :tq]
    shift = torch.arange(0, 8, bits, device=codes.device, dtype=torch.int32)
    x = ((codes.int()[..., None] >> shift) & ((1 << bits) - 1)).flatten(-2)
    if c["sym"]:
        x = torch.where(x >= 1 << (bits - 1), x - (1 << bits), x)
    x = x.float()
    ax, rep = (1, c["g"]) if along_t else (2, c["gv"])
    used = slice(0, tq // c["g"] if along_t else tq)
    if not c["sym"]:
        x = x - s[which + "_zero"][:, used].float().repeat_interleave(rep, ax)
    x = x * s[which + "_scale"][:, used].float().repeat_interleave(rep, ax)
    return torch.cat([x.bfloat16(), s[which + "_resid"][:, :c["nres"]]], 1).float()


def _logits(s):
    """[outer, n * group, T] float32, -inf where a query does not see a token."""
    c = s["case"]
    k = _dequant(s, "k", True)
    O, T, C = k.shape
    n, G = c["n"], c["group"]
    q = s["q"].reshape(c["batch"], n, c["kv_heads"], G, C).transpose(1, 2).reshape(O, n * G, C)
    x = (q.float() @ k.transpose(1, 2)) * C ** -0.5
    t = torch.arange(T, device=x.device)
    last = T - n + torch.arange(n, device=x.device).repeat_interleave(G)
    hidden = (t[None, None] < s["first"][:, None, None]) | (t[None, None] > last[None, :, None])
    return x.masked_fill_(hidden, -math.inf)


def _rows(s, x):
    """[outer, n * group, ...] to the queries' layout [batch, n, heads, ...]."""
    c = s["case"]
    x = x.reshape(c["batch"], c["kv_heads"], c["n"], c["group"], *x.shape[2:]).transpose(1, 2)
    return x.reshape(c["batch"], c["n"], c["kv_heads"] * c["group"], *x.shape[4:])


def _attend(s):
    x = _logits(s)
    top = x.amax(-1, keepdim=True)
    x = x.sub_(top.clamp_min(-3e38)).exp_()
    total = x.sum(-1, keepdim=True)
    out = (x @ _dequant(s, "v", False)) / total.clamp_min(1e-38)
    return _rows(s, out).bfloat16().contiguous(), _rows(s, (top + total.log()).squeeze(-1)).contiguous()


def _weights(s):
    c = s["case"]
    x = _logits(s)
    O, R, T = x.shape
    lse = s["lse"].reshape(c["batch"], c["n"], c["kv_heads"], c["group"]).transpose(1, 2).reshape(O, R, 1)
    return s["scores"][:, :T] + x.sub_(lse.masked_fill(lse == -math.inf, 0.0)).exp_().sum(1)


def _evict(s):
    c = s["case"]
    g, tq, nres = c["g"], c["tq"], c["nres"]
    nb = tq // g
    keep, kept = s["keep"], s["keep"].shape[1]
    recent = min(c["window"], nb)
    score = s["scores"][:, :tq].double().reshape(-1, nb, g).sum(-1)
    order = torch.sort(score[:, :nb - recent], dim=1, descending=True, stable=True).indices[:, :kept - recent]
    newest = torch.arange(nb - recent, nb, device=keep.device).expand(keep.shape[0], recent)
    keep.copy_(torch.cat([order, newest], 1).sort(1).values)
    at = keep.long()
    src = dict((k, s[k]) for k in _STORE if s[k] is not None)
    _take(src, s["dst"], at, g, kept, nb)
    out = s["scores_out"]
    out[:, :kept * g] = s["scores"][:, :tq].reshape(-1, nb, g).gather(1, at[..., None].expand(-1, -1, g)).flatten(1)
    out[:, kept * g:kept * g + nres] = s["scores"][:, tq:tq + nres]
    out[:, kept * g + nres:tq + nres] = 0.0
    pad = s["first"].long()
    s["first_out"].copy_((pad[:, None] - at * g).clamp(0, g).sum(1) + (pad - tq).clamp_min(0))
    return [keep, s["first_out"], out] + [s["dst"][k] for k in _STORE if s[k] is not None]


def _take(src, dst, at, g, kept, nb):
    def one(a, b, per):
        # per: rows of the buffer's middle axis in a block
        row = (at[:, :, None] * per + torch.arange(per, device=at.device)).flatten(1)
        b[:, :kept * per] = a.gather(1, row[..., None].expand(-1, -1, a.shape[2]))
    [one(src[k], dst[k], 1 if k in ("k_scale", "k_zero") else g) for k in src]


# ---- the library -------------------------------------------------------------

def _own_cache(b, s, bufs):
    c = s["case"]
    kw = dict(scale_dtype=b.BF16, residual=128)
    if c["sym"]:
        kq = b.QParams.sym(c["bits"], axis=b.ALONG_T, group=c["g"], **kw)
        vq = b.QParams.sym(c["bits"], axis=b.ALONG_C, group=c["gv"], **kw)
    else:
        kq = b.QParams.asym(c["bits"], 0, (1 << c["bits"]) - 1, axis=b.ALONG_T, group=c["g"], zero_dtype=b.BF16, **kw)
        vq = b.QParams.asym(c["bits"], 0, (1 << c["bits"]) - 1, axis=b.ALONG_C, group=c["gv"], zero_dtype=b.BF16, **kw)
    return b.KVCache(k=(bufs["k_codes"], bufs["k_scale"], bufs["k_zero"], s["k_resid"]),
                     v=(bufs["v_codes"], bufs["v_scale"], bufs["v_zero"], s["v_resid"]),
                     shape=(c["batch"] * c["kv_heads"], c["cap"], c["C"]), kqp=kq, vqp=vq, tq=c["tq"],
                     nres=c["nres"], resid_rows=c["rows"], kv_heads=c["kv_heads"], first=s["first"])


def _own(s):
    from kv_cache_quantization_kvq_gb300 import binding as b
    c = s["case"]
    cache = _own_cache(b, s, s)
    if c["op"] == "attend":
        return b.attend_chunk(s["q"], cache)
    if c["op"] == "weights":
        return b.attend_weights(s["q"], s["lse"], cache, s["scores"])[:, :c["tq"] + c["nres"]]
    dst = _own_cache(b, s, s["dst"])
    dst.first = s["first_out"]
    b.evict_blocks(cache, s["scores"], c["budget"], c["window"], c["g"], dst=dst, scores_out=s["scores_out"],
                   keep=s["keep"])
    return [s["keep"], s["first_out"], s["scores_out"]] + [s["dst"][k] for k in _STORE if s[k] is not None]


def run(state):
    if own:
        return _own(state)
    return {"attend": _attend, "weights": _weights, "evict": _evict}[state["case"]["op"]](state)


# ---- what a pass cannot do without --------------------------------------------

def _pairs(case):
    """Visible (query token, cache token) pairs over all KV slices."""
    T, n, total = case["tq"] + case["nres"], case["n"], 0
    for f in _first(case):
        lo, hi = max(0, T - n + 1 - f), max(0, T - f)       # tokens that the first and the last query see
        total += (lo + hi) * (hi - lo + 1) // 2
    return total


def work(case):
    O, C, bits, tq, nres = case["batch"] * case["kv_heads"], case["C"], case["bits"], case["tq"], case["nres"]
    meta = 2 if case["sym"] else 4
    k_store = tq * C * bits // 8 + tq // case["g"] * C * meta
    v_store = tq * C * bits // 8 + tq * (C // case["gv"]) * meta
    if case["op"] == "evict":
        nb = tq // case["g"]
        kept = min(case["budget"], nb)
        moved = (k_store + v_store) * kept // nb
        return {"bytes": O * (2 * moved + 8 * (tq + nres) + 4 * kept + 8), "flops": 0}
    rows, pairs = O * case["n"] * case["group"], _pairs(case) * case["group"]
    if case["op"] == "attend":
        return {"bytes": O * (k_store + v_store + 4 * nres * C) + rows * (4 * C + 4), "flops": 4 * C * pairs}
    return {"bytes": O * (k_store + 2 * nres * C + 8 * (tq + nres)) + rows * (2 * C + 4), "flops": 2 * C * pairs}


# ---- the definitions in 64 bits ------------------------------------------------

def _value(s, o, which):
    """Slice o's rows in binary64, code by code: s (code - zp) rounded to bf16, then the buffer's rows."""
    c = s["case"]
    per, tq = 8 // c["bits"], c["tq"]
    byte = s[which + "_codes"][o, :tq].long()
    x = torch.empty((tq, c["C"]), dtype=torch.float64, device=byte.device)
    for k in range(per):
        f = torch.div(byte, 2 ** (c["bits"] * k), rounding_mode="floor") % 2 ** c["bits"]
        if c["sym"]:
            f = (f + 2 ** (c["bits"] - 1)) % 2 ** c["bits"] - 2 ** (c["bits"] - 1)
        x[:, k::per] = f.double()
    for name, sign in (("_zero", 0), ("_scale", 1)):
        m = s[which + name]
        if m is None:
            continue
        m = m[o].double()
        if which == "k":
            m = m[torch.arange(tq, device=m.device) // c["g"]]
        else:
            m = m[:tq][:, torch.arange(c["C"], device=m.device) // c["gv"]]
        x = x * m if sign else x - m
    return torch.cat([x.bfloat16().double(), s[which + "_resid"][o, :c["nres"]].double()])


def exact(case, seed):
    if case["op"] != "evict" and _pairs(case) * case["group"] > 6e9:
        return None
    s = prepare(case, seed)
    B, H, G, n, C = case["batch"], case["kv_heads"], case["group"], case["n"], case["C"]
    T = case["tq"] + case["nres"]
    if case["op"] == "evict":
        return _exact_evict(s)
    out = torch.zeros((B, n, H * G, C), dtype=torch.float64, device="cuda")
    lse = torch.full((B, n, H * G), -math.inf, dtype=torch.float64, device="cuda")
    acc = s["scores"][:, :T].double() if case["op"] == "weights" else None
    for o in range(B * H):
        b, h, first = o // H, o % H, _first(case)[o]
        k, v = _value(s, o, "k"), _value(s, o, "v")
        for j in range(G):
            head = h * G + j
            for i0 in range(0, n, 1024):
                q = s["q"][b, i0:i0 + 1024, head].double()
                x = q @ k.T / math.sqrt(C)
                t = torch.arange(T, device="cuda")
                end = T - n + i0 + torch.arange(q.shape[0], device="cuda")
                seen = (t >= first) & (t <= end[:, None])
                x = torch.where(seen, x, -math.inf)
                if case["op"] == "weights":
                    given = s["lse"][b, i0:i0 + 1024, head].double()
                    w = torch.where(seen, torch.exp(x - torch.where(given.isinf(), 0.0, given)[:, None]), 0.0)
                    acc[o] += w.sum(0)
                    continue
                z = torch.logsumexp(x, 1)
                lse[b, i0:i0 + 1024, head] = z
                p = torch.exp(x - torch.where(z.isinf(), 0.0, z)[:, None])
                out[b, i0:i0 + 1024, head] = p @ v
    return acc if case["op"] == "weights" else (out, lse)


def _exact_evict(s):
    c = s["case"]
    g, nb = c["g"], c["tq"] // c["g"]
    kept, recent = min(c["budget"], nb), min(c["window"], nb)
    sc = s["scores"].double().cpu()
    outs = {k: s["dst"][k] for k in _STORE if s[k] is not None}
    keep, first, new = s["keep"], s["first_out"], torch.zeros_like(sc)
    for o in range(sc.shape[0]):
        sums = [float(x) for x in sc[o, :c["tq"]].reshape(nb, g).sum(1)]
        best = sorted(range(nb - recent), key=lambda i: (-sums[i], i))[:kept - recent]
        ids = sorted(best + list(range(nb - recent, nb)))
        keep[o] = torch.tensor(ids, dtype=torch.int32)
        first[o] = sum(min(max(_first(c)[o] - i * g, 0), g) for i in ids) + max(_first(c)[o] - c["tq"], 0)
        rows = torch.tensor([i * g + x for i in ids for x in range(g)])
        new[o, :kept * g] = sc[o, rows]
        new[o, kept * g:kept * g + c["nres"]] = sc[o, c["tq"]:c["tq"] + c["nres"]]
        for k, d in outs.items():
            r = torch.tensor(ids) if k in ("k_scale", "k_zero") else rows
            d[o, :len(r)] = s[k][o][r.to(d.device)]
    return [keep, first, new] + [outs[k] for k in _STORE if s[k] is not None]
